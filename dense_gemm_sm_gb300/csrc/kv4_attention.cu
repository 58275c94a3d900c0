// kv4_attention.cu -- attention of the newest tokens of each sequence over the paged 4-bit
// cache: for query i of sequence b (its position is len_b - Lq + i),
//   O = sum_j softmax_j(scale * q . K_j) V_j   over the keys j <= len_b - Lq + i,
// K_j = kz_j + ks_j kc_j and V_j = vz_j + vs_j vc_j (codes kc, vc in 0..15 per element, one scale
// and zero per row).  A query that sees no key gets 0.
//
// Bytes bound it: d + 8 bytes of cache per (token, head) against 4 d flops per query of the
// group.  So the codes go from HBM to the tensor cores' operand registers with as few
// instructions as can be:
//   * keys (and V's columns) are the 16 rows of an mma.m16n8k16 and the queries its 8 columns:
//     one token of up to 8 query heads per cache head fills the tile, and a dequantised
//     fragment serves all queries.  (tcgen05 would want the expanded operand written to shared
//     or tensor memory first, for products that are a few percent of the time here.)
//   * a code n becomes the BF16 number 128 + n by one AND-OR on the packed word (two codes of
//     one 32-bit register at a time); the 128 is taken out in FP32 afterwards, with the row's
//     scale and zero:
//       q . K_j = ks_j (q . (128 + kc_j)) + (kz_j - 128 ks_j) sum(q),
//       O = sum_j P_j (128 + vc_j) - 136 sum_j P_j + sum_j p_j (vz_j + 8 vs_j),
//     P_j = bf16(p_j vs_j).  The middle sum takes the rounded P_j: what the rounding of P
//     multiplies is vc_j - 8, V's deviation from the middle of its range and not from its
//     minimum (64 ragged sequences of normal rows: 0.0011 of O in the mean square, 0.0031 without).
//   * the order of d in the first product and of keys in the second is free: K rows are read
//     as they lie (a lane 16 bytes, two key rows), V's codes lie in the cache in fragment order.
//   * P goes from the first product's output layout to the second's operand layout by
//     movmatrix, in registers.
// Work: units of 32 keys of all (sequence, cache head, query block) items, in one row, cut evenly
// over the CTAs (one per SM) and each CTA's share over its warps, whatever the lengths: a warp
// walks its units with its own ring of bulk copies (one per 16-token record, so pages of any
// multiple of 16 do) and writes the items that lie whole in its share.  An item cut between warps of a CTA is joined
// once, at the CTA's end, through shared memory; one cut between CTAs by the last of them to
// arrive, in CTA order (so results do not depend on arrival), of very many CTAs in two steps.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

constexpr int kMaxCtas = 160;   // CTAs that the workspace has room for
// A CTA is given at least this many units, so that small calls use fewer CTAs and joins.
constexpr int kMinUnits = 4;
// Items of up to this many units are one CTA's, which mostly saves the join of two (8 cache heads
// of 128, 8 queries each; us with 0, 16, 32, 64 here: 16 x 512 keys 12.2, 9.1, 9.1, 9.1;
// 100 x 1024 32.5, 32.6, 30.4, 30.3; 8 x 1024 of four queries 31.8, 31.8, 20.3, 20.3;
// 1 x 1024 8.9, 8.9, 10.2, 10.2; 1 x 2048 9.8, 9.8, 9.8, 13.4).  With a few more items than one or
// two a CTA the longest share is then up to twice the even one; even there the joins saved are
// worth it, but for 9 query rows and more, where it costs up to 5 % (items of 32 units, us with 0 and
// 32 here, at 152, 160, 200 and 320 items: 4 rows 10.2, 10.2; 14.2, 13.2; 14.9, 13.3; 18.0, 17.5; 16 rows
// 12.8, 12.8; 18.6, 19.0; 21.4, 19.2; 25.6, 26.3; 32 rows 20.5, 20.5; 31.6, 32.7; 37.0, 33.0; 44.5, 46.4).
constexpr int kWhole = 32;
// The reference that weights are taken against (2^(score - reference)) follows the running
// maximum only when that has outgrown it by this much: weights stay below 2^8, which FP32 sums
// and BF16's exponent carry as well as weights below 1, and most steps scale nothing.
constexpr float kSlack = 8.f;
// An item of very many CTAs is joined in two steps, this many neighbours first.
constexpr uint32_t kTeam = 12;
constexpr int kTeams = 2 * ((kMaxCtas + kTeam - 1) / kTeam);  // places of their sums and counters
constexpr int64_t kCounterBytes = 1024;  // ticket counters of the CTAs and the teams, then the parts
static_assert((kMaxCtas + kTeams) * 4 <= kCounterBytes, "counters");

template <int D, int NT>
struct Cfg {
  static constexpr int kUnit = 32;                              // keys of a unit
  static constexpr int kRecs = kUnit / kKv4Tokens;
  static constexpr int kRec = kv4_record_bytes(D);
  static constexpr int kUnitBytes = kRecs * kRec;
  static constexpr int kWarps = NT == 1 ? 15 : 7;               // that compute; one more issues the copies
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kStages = NT == 1 && D == 128 ? 3 : 4;
  static constexpr int kRing = kWarps * kStages * kUnitBytes;
  static constexpr int kRows = 8 * NT;
  // A part: rows of outputs, then the rows' maxima and their sums of weights.  Rows of 128 are
  // padded: a warp's 16-byte stores would otherwise all start in two banks (one 8192-token
  // sequence 12.4 us, 11.3 so; rows of 64 measured no better padded).
  static constexpr int kPitch = D == 128 ? D + 4 : D;
  static constexpr int kTop = kRows * kPitch, kSum = kTop + kRows;
  static constexpr int kPart = kSum + kRows;
  static constexpr int kQ = NT == 4 ? NT * (D / 16) * 32 * 8 : 0;  // a warp's Q fragments (registers otherwise)
  static constexpr int kSmem = kRing + kWarps * kQ;
  static_assert(kWarps * kPart * 4 <= kRing, "the warps' last parts take the ring's place");
  static_assert(kSmem + 4096 <= 227 * 1024, "shared memory, with the static part");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Codes n of the pair of halves' n-th nibbles -> BF16 pair 128 + code.  Mask and offset come in
// registers: as two constants the AND and the OR are two instructions, and the logic pipe, which
// takes one every other cycle, is what the kernel runs into (8 x 66k tokens: 921 instructions of
// a 64-key unit on it, 541 of them these).
struct Magic {
  uint32_t mask, offset;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(offset));
  }
  template <int N>
  __device__ __forceinline__ uint32_t expand(uint32_t w) const {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w >> (4 * N)), "r"(mask), "r"(offset));  // (a & b) | c
    return d;
  }
};

template <int WORDS>
__device__ __forceinline__ void lds(uint32_t a, uint32_t (&w)[WORDS]) {
  if (WORDS == 4) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[WORDS - 2]), "=r"(w[WORDS - 1])
                 : "r"(a));
  } else {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  }
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint32_t lds1(uint32_t a) {
  uint32_t w;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(a));
  return w;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t take_ticket(uint32_t* a) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a) : "memory");
  return old;
}

// Units cut evenly over workers, the first `rem` of them one unit longer.  Units and workers
// fit 31 bits.
struct Split {
  uint32_t q, rem;
  __device__ __forceinline__ Split(uint32_t units, uint32_t workers) : q(units / workers), rem(units - q * workers) {}
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return c * q + (c < rem ? c : rem); }
  __device__ __forceinline__ uint32_t worker(uint32_t x) const {  // that has unit x
    const uint32_t long_units = rem * (q + 1);
    return x < long_units ? x / (q + 1) : rem + (x - long_units) / q;
  }
};

// Position in the row of all units: unit r is unit u of item `item` of sequence b.
struct Walk {
  uint32_t r, b;
  int32_t len, units, item, u;
};

// An item that a warp has a part of.
struct Cut {
  uint32_t b, first;  // sequence, the item's first unit
  int32_t item, units;
};

// A running softmax-weighted sum of parts: maximum, sum of weights, four outputs.
struct Sum {
  float m = -INFINITY, l = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  // Adds N parts against their common maximum: their weights do not wait for one another.  Parts
  // without a maximum saw no key, or scores that are all NaN: those sums are NaN and stay it.
  template <int N>
  __device__ __forceinline__ void add(const float (&mk)[N], const float (&lk)[N], const float4 (&x)[N]) {
    float top = m;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, mk[i]);
    const float ref = top > -INFINITY ? top : 0.f;
    const float a = ex2(m - ref);
    m = top;
    l *= a;
    v = make_float4(v.x * a, v.y * a, v.z * a, v.w * a);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float b = ex2(mk[i] - ref);
      l = fmaf(lk[i], b, l);
      v = make_float4(fmaf(x[i].x, b, v.x), fmaf(x[i].y, b, v.y), fmaf(x[i].z, b, v.z), fmaf(x[i].w, b, v.w));
    }
  }
  __device__ __forceinline__ uint2 value() const {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    return make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
  }
};

template <int D, int NT>
struct Shared {
  static constexpr int kWarps = Cfg<D, NT>::kWarps;
  uint64_t full[kWarps * 4], empty[kWarps * 4];
  uint32_t mask[kWarps * 4];   // records of the stage that were copied
  Walk start[kWarps];
  Cut head[kWarps], tail[kWarps];
  uint8_t has_head[kWarps], has_tail[kWarps];
  int32_t last[2];             // runs of items of other CTAs too, for which this CTA came last; -1: none
  int32_t runs;
  bool ends[2];                // the step of its join is the item's last
  struct Run {
    int8_t first, last, head;  // warps of its tails (first < 0: none) and its head (< 0: none)
    int8_t slot;               // -1: the item is this CTA's alone, else the CTA's part that this is
  } run[kWarps + 1];
  // Where a row of a run's item goes in O; -1: no such row.
  int64_t row_at[kWarps + 1][8 * NT];
  uint32_t issued[kWarps];     // stages of a ring that were filled, over the whole call
  uint32_t abort;
};

// TREE: a query sees, of the sequence's newest tokens, those that its mask names, and a sequence may
// have fewer than Lq queries; the others' rows are zeros.
template <int D, int NT, bool TREE>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    kv4_attention_kernel(const Kv4AttnParams p, const int qblocks) {
  using C = Cfg<D, NT>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads, kUnit = C::kUnit, kRecs = C::kRecs;
  constexpr int KS = D / 16;       // k steps of the first product
  constexpr int MT = D / 16;       // m tiles of the second
  constexpr int W = D / 32;        // words of a lane's share of a row
  constexpr uint32_t kOnes = 0x3F803F80u;
  const Magic magic;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared<D, NT> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kUnitBytes;
  const uint32_t qfrag = smem_u32(smem) + C::kRing + warp * C::kQ;

  if (lane == 0 && warp < kWarps)
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&sh.full[warp * 4 + s]), 1);
      mbar_init(smem_u32(&sh.empty[warp * 4 + s]), 1);
    }
  if (tid == 0) sh.abort = 0;
  if (tid < 2) sh.last[tid] = -1;
  if (tid < kWarps) sh.has_head[tid] = sh.has_tail[tid] = 0, sh.issued[tid] = 0;
  fence_barrier_init();
  __syncthreads();
  pdl_trigger();
  pdl_wait();

  const int32_t cap = static_cast<int32_t>(p.ldt * p.page_size);
  auto nodes_of = [&](uint32_t b) -> int32_t {  // a tree's queries
    const int32_t n = p.nodes ? p.nodes[b] : static_cast<int32_t>(p.Lq);
    return min(max(n, 0), static_cast<int32_t>(p.Lq));
  };
  // A tree without a query is no work, whatever its context (8 contexts of 65000 tokens without one beside 8 of
  // 500 tokens with two: 107 us as work, 9.5 so).  Both numbers are asked for at once.
  auto len_of = [&](uint32_t b) -> int32_t {
    const int32_t n = p.lens[b], queries = TREE ? nodes_of(b) : 1;
    return queries == 0 ? 0 : min(max(n, 0), cap);
  };
  const int ips = p.heads * qblocks;  // items of a sequence
  const int rows_all = static_cast<int>(p.Lq) * p.group;
  const uint32_t batch = static_cast<uint32_t>(p.batch);

  // ---- every warp adds up the units for itself; a lane takes a run of sequences, and keeps the
  // units of the first few
  constexpr int kKept = 4;
  const uint32_t per = (batch + 31) / 32, b_lo = lane * per, b_hi = min(b_lo + per, batch);
  auto units_of = [&](uint32_t b) {
    const int32_t n = p.lens[b], queries = TREE && p.nodes ? p.nodes[b] : 1;
    if (blockIdx.x == 0 && (n < 0 || n > cap || queries < 0 || queries > p.Lq)) atomicCAS(p.index_word, 0u, kDevBadIndex);
    return queries <= 0 ? 0u : static_cast<uint32_t>(min(max(n, 0), cap) + kUnit - 1) / kUnit;
  };
  uint32_t kept[kKept], mine = 0;
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    kept[i] = b_lo + i < b_hi ? units_of(b_lo + i) : 0;
    mine += kept[i];
  }
#pragma unroll 1
  for (uint32_t b = b_lo + kKept; b < b_hi; ++b) mine += units_of(b);
  mine *= ips;
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  const uint32_t total = __shfl_sync(~0u, incl, 31);

  // ---- sequences without a token or a query
#pragma unroll 1
  for (uint32_t b = blockIdx.x; b < batch; b += gridDim.x) {
    if (len_of(b) > 0) continue;
    const int words = p.group * p.heads * (D / 8);  // of 16 bytes, a query
#pragma unroll 1
    for (int64_t i = tid; i < p.Lq * words; i += kThreads)
      *reinterpret_cast<uint4*>(p.O + b * p.strideO + i / words * p.ldo + i % words * 8) = make_uint4(0, 0, 0, 0);
  }
  const uint32_t ctas = min((total + kMinUnits - 1) / kMinUnits, gridDim.x);
  if (blockIdx.x >= ctas) return;  // whole CTAs
  const Split split(total, ctas);

  // Where unit r < total lies (all lanes): the lane whose sequences hold it finds the sequence and
  // what lies before it there.
  auto locate = [&](uint32_t r) {
    const int owner = __ffs(__ballot_sync(~0u, r < incl)) - 1;
    uint32_t at = incl - mine, b0 = b_lo, units = 0;
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < kKept; ++i)
        if (units == 0) {
          const uint32_t n = kept[i] * ips;
          if (r < at + n) {
            units = kept[i];
          } else {
            at += n;
            ++b0;
          }
        }
#pragma unroll 1
      while (units == 0) {
        const uint32_t here = static_cast<uint32_t>(len_of(b0) + kUnit - 1) / kUnit;
        if (r < at + here * ips) {
          units = here;
        } else {
          at += here * ips;
          ++b0;
        }
      }
    }
    Walk w;
    w.r = r;
    w.b = __shfl_sync(~0u, b0, owner);
    w.units = __shfl_sync(~0u, units, owner);
    const uint32_t off = r - __shfl_sync(~0u, at, owner);
    w.item = off / static_cast<uint32_t>(w.units);
    w.u = off - w.item * w.units;
    return w;
  };
  // The CTAs' shares: even, but a border inside an item of up to kWhole units moves to the item's
  // nearer end.  (Borders inside longer items stay, so the CTAs of such an item are the even
  // cut's.)
  auto border = [&](uint32_t c) {
    const uint32_t r = split.start(c);
    if (c == 0 || c == ctas) return r;
    const Walk w = locate(r);
    return w.units > kWhole ? r : 2 * w.u < w.units ? r - w.u : r - w.u + w.units;
  };
  const uint32_t cta_r0 = border(blockIdx.x), cta_r1 = border(blockIdx.x + 1);
  // The units of this warp, and of the warp that a lane of the copying warp works for.
  const bool copies = warp == kWarps;
  const uint32_t me = blockIdx.x * kWarps + warp;
  const Split share(cta_r1 - cta_r0, kWarps);
  const uint32_t w0 = copies ? min(lane, kWarps - 1) : warp;
  const uint32_t r0 = cta_r0 + share.start(w0), r1 = cta_r0 + share.start(w0 + 1);

  auto move_to = [&](Walk& w, uint32_t r) {  // r < total
    int32_t d = static_cast<int32_t>(r - w.r);
    w.r = r;
#pragma unroll 1
    while (d >= w.units - w.u) {
      d -= w.units - w.u;
      w.u = 0;
      if (++w.item == ips) {
        w.item = 0;
        do {
          ++w.b;
          w.len = len_of(w.b);
        } while (w.len == 0);
        w.units = (w.len + kUnit - 1) / kUnit;
      }
    }
    w.u += d;
  };

  Walk seg;
  if (!copies && r0 < r1) {
    seg = locate(r0);
    seg.len = len_of(seg.b);
    if (lane == 0) sh.start[warp] = seg;
  }
  __syncthreads();

  if (copies) {
    // ---- a lane fills the ring of the warp of its number: the bookkeeping of all rings is done
    // once for all of them, not in every computing warp (where it took a tenth of the time)
    if (lane < kWarps && r0 < r1) {
      Walk at = sh.start[lane];
      const uint32_t to = smem_u32(smem) + lane * C::kStages * C::kUnitBytes;
      const int32_t page_recs = p.page_size / kKv4Tokens;
      int nrec;
      uint32_t rec_in[kRecs];
      int32_t page[kRecs];
      auto look_up = [&]() {  // the pages of the next unit's records
        const uint32_t n = static_cast<uint32_t>(at.u) * kRecs;
        nrec = (at.len - at.u * kUnit + kKv4Tokens - 1) / kKv4Tokens;
        nrec = nrec < kRecs ? nrec : kRecs;
#pragma unroll
        for (int i = 0; i < kRecs; ++i) {
          // Records are whole: the page of record n is n / (page_size / 16), by multiplication.
          const uint32_t pi = p.page_magic ? __umulhi(n + i, p.page_magic) : n + i;
          rec_in[i] = n + i - pi * page_recs;
          page[i] = i < nrec ? p.table[static_cast<int64_t>(at.b) * p.ldt + pi] : -1;
        }
      };
      look_up();
      uint32_t put = 0;  // slot, and its phase in bit 8
      uint32_t fresh = C::kStages;  // slots never used
      uint64_t since = 0;
      uint32_t issued = 0;
#pragma unroll 1
      for (;;) {
        const uint32_t s = put & 255u;
        if (fresh == 0 && !mbar_test(smem_u32(&sh.empty[lane * 4 + s]), (put >> 8) ^ 1u)) {
          __nanosleep(40);
          const uint64_t now = globaltimer_ns();
          if (since == 0) since = now;
          if (now - since > kWaitLimitNs || *static_cast<volatile uint32_t*>(&sh.abort)) {
            sh.abort = 1;
            atomicCAS(p.status, 0u, kDevTimeoutProducer);
            break;
          }
          continue;
        }
        since = 0;
        if (fresh) --fresh;
        const uint32_t bar = smem_u32(&sh.full[lane * 4 + s]);
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < kRecs; ++i) {
          if (page[i] >= 0 && page[i] < p.pages) mask |= 1u << i;
          else if (i < nrec) atomicCAS(p.index_word, 0u, kDevBadIndex);
        }
        sh.mask[lane * 4 + s] = mask;
        mbar_arrive_expect_tx(bar, __popc(mask) * C::kRec);
        const int64_t head = at.item / qblocks;
        // Pages of whole units: one copy; otherwise one a record.
#pragma unroll
        for (int i = 0; i < kRecs; ++i) {
          if (!((mask >> i) & 1u) || (p.one_copy && i > 0)) continue;
          const uint8_t* src = p.data + ((static_cast<int64_t>(page[i]) * p.heads + head) * page_recs + rec_in[i]) * C::kRec;
          bulk_load(to + s * C::kUnitBytes + i * C::kRec, src, p.one_copy ? nrec * C::kRec : C::kRec, bar);
        }
        put = s + 1 == C::kStages ? (put & 256u) ^ 256u : put + 1;
        ++issued;
        if (at.r + 1 >= r1) break;
        move_to(at, at.r + 1);
        look_up();
      }
      sh.issued[lane] = issued;
    }
  } else if (r0 < r1) {
    uint32_t got = 0;  // stage in use: the slot, and its phase in bit 8
    // ---- segments: this warp's piece of one item after the other
#pragma unroll 1
    for (;;) {
      const int32_t n = min(seg.units - seg.u, static_cast<int32_t>(r1 - seg.r));
      const int head = seg.item / qblocks;
      const int row0 = (seg.item - head * qblocks) * C::kRows;
      const uint16_t* qbase = p.Q + static_cast<int64_t>(seg.b) * p.strideQ + static_cast<int64_t>(head) * p.group * D;
      const int nodes = TREE ? nodes_of(seg.b) : 0;
      const int live = TREE ? nodes * p.group : rows_all;  // query rows that see anything
      // The keys before this one are visible to all of them.
      const int shared_keys = seg.len - (TREE ? nodes : static_cast<int>(p.Lq) - 1);

      // Q fragments: lane (g, t) takes query row g's elements [t d/4, + d/4).
      uint32_t qf[NT <= 2 ? NT : 1][KS][2];
      float qsum[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + nt * 8 + g;
        uint4 w[W];
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = make_uint4(0, 0, 0, 0);
        if (row < live) {
          const uint4* src = reinterpret_cast<const uint4*>(qbase + static_cast<int64_t>(row / p.group) * p.ldq +
                                                            (row % p.group) * D + t * (D / 4));
#pragma unroll
          for (int j = 0; j < W; ++j) w[j] = __ldg(src + j);
        }
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t f[4] = {__byte_perm(w[j].x, w[j].z, 0x5410), __byte_perm(w[j].x, w[j].z, 0x7632),
                                 __byte_perm(w[j].y, w[j].w, 0x5410), __byte_perm(w[j].y, w[j].w, 0x7632)};
#pragma unroll
          for (int i = 0; i < 4; ++i) sum += lo_of(f[i]) + hi_of(f[i]);
          if constexpr (NT <= 2) {
            qf[nt][2 * j][0] = f[0];
            qf[nt][2 * j][1] = f[1];
            qf[nt][2 * j + 1][0] = f[2];
            qf[nt][2 * j + 1][1] = f[3];
          } else {  // read back by the same lane only
            const uint32_t a = qfrag + ((nt * KS + 2 * j) * 32 + lane) * 8;
            asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a), "r"(f[0]), "r"(f[1]) : "memory");
            asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a + 256), "r"(f[2]), "r"(f[3]) : "memory");
          }
        }
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
        // An infinite sum becomes NaN: codes and zeros may both pull all scores to -Inf, and a row without a score
        // above that is one that sees no key.
        sum = fmaf(0.f, sum, sum);
#pragma unroll
        for (int e = 0; e < 2; ++e) qsum[nt][e] = __shfl_sync(~0u, sum, (2 * t + e) * 4);
      }

      float o[NT][MT][4], m[NT][2], l[NT][2], z[NT][2];
      float ps[NT][4];  // column sums of the rounded P, by a product with ones
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = -INFINITY;
          l[nt][e] = z[nt][e] = 0.f;
          ps[nt][e] = ps[nt][2 + e] = 0.f;
        }
      }

      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const uint32_t slot = got & 255u;
        ok = __all_sync(~0u, mbar_wait(smem_u32(&sh.full[warp * 4 + slot]), got >> 8, &sh.abort, p.status, kDevTimeoutMma));
        if (!ok) break;
        const uint32_t have = sh.mask[warp * 4 + slot];
        {
          const uint32_t st = ring + slot * C::kUnitBytes;
          const int key0 = (seg.u + j) * kUnit;
          const bool whole = have == (1u << kRecs) - 1 && key0 + kUnit <= shared_keys;
          // ---- S = K Q^T
          float sc[kRecs][NT][4];
#pragma unroll
          for (int r = 0; r < kRecs; ++r) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[r][nt][e] = 0.f;
            uint32_t ka[W], kb[W];
            lds(st + r * C::kRec + g * (D / 2) + t * (D / 8), ka);
            lds(st + r * C::kRec + (g + 8) * (D / 2) + t * (D / 8), kb);
#pragma unroll
            for (int w = 0; w < W; ++w) {
              const uint32_t a[4] = {magic.expand<0>(ka[w]), magic.expand<1>(ka[w]), magic.expand<2>(ka[w]), magic.expand<3>(ka[w])};
              const uint32_t b[4] = {magic.expand<0>(kb[w]), magic.expand<1>(kb[w]), magic.expand<2>(kb[w]), magic.expand<3>(kb[w])};
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  uint32_t q0, q1;
                  if constexpr (NT <= 2) {
                    q0 = qf[nt][2 * w + i][0];
                    q1 = qf[nt][2 * w + i][1];
                  } else {
                    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                                 : "=r"(q0), "=r"(q1)
                                 : "r"(qfrag + ((nt * KS + 2 * w + i) * 32 + lane) * 8));
                  }
                  mma_bf16(sc[r][nt], a[2 * i], b[2 * i], a[2 * i + 1], b[2 * i + 1], q0, q1);
                }
            }
          }
          // ---- scores in log2 units
#pragma unroll
          for (int r = 0; r < kRecs; ++r) {
            const uint32_t pa = lds1(st + r * C::kRec + 16 * D + g * 4), pb = lds1(st + r * C::kRec + 16 * D + (g + 8) * 4);
            const float s0 = lo_of(pa), s1 = lo_of(pb);
            const float m0 = s0 * p.c_log2, m1 = s1 * p.c_log2;
            const float a0 = fmaf(-128.f, s0, hi_of(pa)) * p.c_log2, a1 = fmaf(-128.f, s1, hi_of(pb)) * p.c_log2;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                sc[r][nt][e] = fmaf(sc[r][nt][e], m0, a0 * qsum[nt][e]);
                sc[r][nt][2 + e] = fmaf(sc[r][nt][2 + e], m1, a1 * qsum[nt][e]);
              }
          }
          uint32_t vp[kRecs][2];
#pragma unroll
          for (int r = 0; r < kRecs; ++r) {
            vp[r][0] = lds1(st + r * C::kRec + 16 * D + 64 + g * 4);
            vp[r][1] = lds1(st + r * C::kRec + 16 * D + 64 + (g + 8) * 4);
          }
          if (!whole) {  // the last units, and pages outside the cache
            asm volatile("" ::: "memory");  // a branch: few steps come here
            uint64_t see[NT][2];  // the tree's nodes that a query sees
            if constexpr (TREE) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int row = row0 + nt * 8 + 2 * t + e;
                  see[nt][e] = row < live ? p.mask[static_cast<int64_t>(seg.b) * p.Lq + row / p.group] : 0;
                }
            }
#pragma unroll
            for (int r = 0; r < kRecs; ++r)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int k = key0 + r * kKv4Tokens + 8 * i + g;
                const bool in = ((have >> r) & 1u) && k < seg.len;
                // A row that no query sees may hold anything.  A query that does not see one that others may see
                // weighs it by 0: V's numbers that are not finite become 0 there, and scores NaN for those that see it.
                if (!in) vp[r][i] = 0;
                const bool wild = k >= shared_keys && !(fabsf(fmaf(8.f, lo_of(vp[r][i]), hi_of(vp[r][i]))) < INFINITY);
                if (wild) vp[r][i] = 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    bool seen;
                    if constexpr (TREE) {
                      const int node = k - shared_keys;  // below 64 where `in`
                      seen = node < 0 || ((see[nt][e] >> (node & 63)) & 1u);
                    } else {
                      seen = k <= seg.len - static_cast<int>(p.Lq) + (row0 + nt * 8 + 2 * t + e) / p.group;
                    }
                    if (!in || !seen) sc[r][nt][2 * i + e] = -INFINITY;
                    else if (wild) sc[r][nt][2 * i + e] = __uint_as_float(0x7FC00000u);
                  }
              }
          }
          // ---- running maximum (a column's keys lie across the lanes' g)
          float use[NT][2];
          bool grew = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = fmaxf(sc[0][nt][e], sc[0][nt][2 + e]);
#pragma unroll
              for (int r = 1; r < kRecs; ++r) v = fmaxf(v, fmaxf(sc[r][nt][e], sc[r][nt][2 + e]));
              v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
              v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
              v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
              grew |= v > m[nt][e] + kSlack;
              use[nt][e] = fmaxf(m[nt][e], v);
            }
          if (__any_sync(~0u, grew)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // Nothing seen so far (-inf) has nothing to scale: the factor only must not be NaN.
                const float f = m[nt][e] > -INFINITY ? ex2(m[nt][e] - use[nt][e]) : 0.f;
                m[nt][e] = use[nt][e];
                l[nt][e] *= f;
                z[nt][e] *= f;
                ps[nt][e] *= f;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                  o[nt][i][e] *= f;
                  o[nt][i][2 + e] *= f;
                }
              }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) use[nt][e] = m[nt][e] > -INFINITY ? m[nt][e] : 0.f;
          // ---- P, and O += V^T P^T record by record
#pragma unroll
          for (int r = 0; r < kRecs; ++r) {
            const float s0 = lo_of(vp[r][0]), s1 = lo_of(vp[r][1]);
            const float z0 = fmaf(8.f, s0, hi_of(vp[r][0])), z1 = fmaf(8.f, s1, hi_of(vp[r][1]));
            uint32_t b0[NT], b1[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = ex2(sc[r][nt][e] - use[nt][e & 1]);
              l[nt][0] += w[0] + w[2];
              l[nt][1] += w[1] + w[3];
              z[nt][0] = fmaf(w[0], z0, fmaf(w[2], z1, z[nt][0]));
              z[nt][1] = fmaf(w[1], z0, fmaf(w[3], z1, z[nt][1]));
              b0[nt] = transpose8x8(pack2(w[0] * s0, w[1] * s0));
              b1[nt] = transpose8x8(pack2(w[2] * s1, w[3] * s1));
              mma_bf16(ps[nt], kOnes, kOnes, kOnes, kOnes, b0[nt], b1[nt]);
            }
            uint32_t va[W], vb[W];
            lds(st + r * C::kRec + 8 * D + lane * (D / 8), va);
            lds(st + r * C::kRec + 8 * D + (32 + lane) * (D / 8), vb);
#pragma unroll
            for (int w = 0; w < W; ++w) {
              const uint32_t a[4] = {magic.expand<0>(va[w]), magic.expand<1>(va[w]), magic.expand<2>(va[w]), magic.expand<3>(va[w])};
              const uint32_t b[4] = {magic.expand<0>(vb[w]), magic.expand<1>(vb[w]), magic.expand<2>(vb[w]), magic.expand<3>(vb[w])};
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_bf16(o[nt][2 * w + i], a[2 * i], a[2 * i + 1], b[2 * i], b[2 * i + 1], b0[nt], b1[nt]);
            }
          }
        }
        __syncwarp();  // all lanes have read the stage
        if (lane == 0 && p.fault != 1) mbar_arrive(smem_u32(&sh.empty[warp * 4 + slot]));
        got = slot + 1 == C::kStages ? (got & 256u) ^ 256u : got + 1;
      }
      if (!ok) break;  // given up: nothing of this piece is kept

      // ---- the segment's sums; a whole item is written, a part kept for the join
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], x);
            z[nt][e] += __shfl_xor_sync(~0u, z[nt][e], x);
          }
          z[nt][e] = fmaf(-136.f, ps[nt][e], z[nt][e]);
          if (TREE && row0 + nt * 8 + 2 * t + e >= live) {  // no query: nothing summed
            l[nt][e] = z[nt][e] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[nt][i][e] = o[nt][i][2 + e] = 0.f;
          }
        }
      const bool ends = seg.u + n == seg.units;
      if (seg.u == 0 && ends) {
        uint16_t* obase = p.O + static_cast<int64_t>(seg.b) * p.strideO + static_cast<int64_t>(head) * p.group * D + g * (D / 8);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = row0 + nt * 8 + 2 * t + e;
            const float inv = l[nt][e] > 0.f ? 1.f / l[nt][e] : 0.f;
            uint32_t w[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i)
              w[i] = pack2((o[nt][i][e] + z[nt][e]) * inv, (o[nt][i][2 + e] + z[nt][e]) * inv);
            if (row < rows_all) {
              uint4* dst = reinterpret_cast<uint4*>(obase + static_cast<int64_t>(row / p.group) * p.ldo + row % p.group * D);
#pragma unroll
              for (int i = 0; i < MT / 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
          }
      } else {
        // The warp's last piece takes its ring's place, an earlier one (which ends an item that
        // another warp began) a place in the workspace.
        float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kCounterBytes) +
                      static_cast<int64_t>(me) * C::kPart;
        if (seg.r + n == r1) {
          __syncwarp();
          part = reinterpret_cast<float*>(smem + warp * C::kStages * C::kUnitBytes);
          static_assert(C::kPart * 4 <= C::kStages * C::kUnitBytes, "a warp's part fits its own ring");
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = nt * 8 + 2 * t + e;
            float4* dst = reinterpret_cast<float4*>(part + row * C::kPitch + g * (D / 8));
#pragma unroll
            for (int i = 0; i < MT / 2; ++i)
              dst[i] = make_float4(o[nt][2 * i][e] + z[nt][e], o[nt][2 * i][2 + e] + z[nt][e],
                                   o[nt][2 * i + 1][e] + z[nt][e], o[nt][2 * i + 1][2 + e] + z[nt][e]);
            if (g == 0) {
              part[C::kTop + row] = m[nt][e];
              part[C::kSum + row] = l[nt][e];
            }
          }
        if (lane == 0) {
          Cut* cut = ends ? &sh.head[warp] : &sh.tail[warp];
          cut->b = seg.b;
          cut->first = seg.r - seg.u;
          cut->item = seg.item;
          cut->units = seg.units;
          (ends ? sh.has_head[warp] : sh.has_tail[warp]) = seg.r + n == r1 ? 2 : 1;  // 2: in the ring's place
        }
      }
      if (seg.r + n >= r1) break;
      move_to(seg, seg.r + n);
    }
  }
  __syncthreads();
  if (sh.abort) {
    // Some wait of this CTA ran out: its results are void, no ticket is taken.  What it copies still
    // lands in its own rings before it ends.
    if (lane == 0 && !copies) {
      const uint32_t issued = sh.issued[warp];
      uint32_t never = 0;
      for (uint32_t i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
        mbar_wait(smem_u32(&sh.full[warp * 4 + i % C::kStages]), i / C::kStages & 1u, &never, p.status, kDevTimeoutDrain);
    }
    return;
  }

  // ---- join: the parts in the order of their units are head 0, tail 0, head 1, tail 1, ...; a
  // tail and what follows it, up to the next head, are one item: a run.
  auto tail_part = [&](int w) { return reinterpret_cast<const float*>(smem + w * C::kStages * C::kUnitBytes); };
  auto head_part = [&](int w) {
    return sh.has_head[w] == 2 ? tail_part(w)
                               : reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.ws) + kCounterBytes) +
                                     (static_cast<int64_t>(blockIdx.x) * kWarps + w) * C::kPart;
  };
  float* cta_parts = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kCounterBytes) +
                     static_cast<int64_t>(kMaxCtas) * kWarps * C::kPart;
  // Element offset in O of a row of the item, -1 past its rows.
  auto row_of = [&](const Cut& cut, int row) -> int64_t {
    const int head = cut.item / qblocks, rr = (cut.item - head * qblocks) * C::kRows + row;
    if (rr >= rows_all) return -1;
    return static_cast<int64_t>(cut.b) * p.strideO + static_cast<int64_t>(rr / p.group) * p.ldo +
           (static_cast<int64_t>(head) * p.group + rr % p.group) * D;
  };
  if (warp == 0) {
    // Bit w: warp w has a tail, a head.  A run ends at a head, or (the last) after the last
    // warp; it begins at the first tail after the end of the one before, or is a head alone.
    const uint32_t tails = __ballot_sync(~0u, lane < kWarps && sh.has_tail[lane < kWarps ? lane : 0]);
    const uint32_t heads = __ballot_sync(~0u, lane < kWarps && sh.has_head[lane < kWarps ? lane : 0]);
    const uint32_t upto = (2u << lane) - 1;  // warps 0 .. lane
    const bool is_head = (heads >> lane) & 1u;
    // The previous head's own tail belongs to the run that follows it.
    const uint32_t before = heads & (upto >> 1);
    const uint32_t own = tails & ~(before ? (1u << (31 - __clz(before))) - 1 : 0u);
    const uint32_t run_tails = own & (upto >> 1);
    if (is_head) {
      auto& run = sh.run[__popc(before)];
      run.first = static_cast<int8_t>(__ffs(run_tails) - 1);
      run.last = static_cast<int8_t>(31 - __clz(run_tails));
      run.head = static_cast<int8_t>(lane);
    }
    if (lane == kWarps) {  // what is left after the last head
      auto& run = sh.run[__popc(heads)];
      run.first = static_cast<int8_t>(__ffs(own) - 1);
      run.last = static_cast<int8_t>(31 - __clz(own));
      run.head = -1;
      sh.runs = __popc(heads) + (own ? 1 : 0);
    }
  }
  __syncthreads();
  // What an output needs of its run and row is worked out once: with the divisions in every
  // output the join of a batch of ragged sequences took 8 us of its 48.
#pragma unroll 1
  for (int i = tid; i < sh.runs * C::kRows; i += kThreads) {
    auto& run = sh.run[i / C::kRows];
    const Cut& cut = run.first >= 0 ? sh.tail[run.first] : sh.head[run.head];
    sh.row_at[i / C::kRows][i % C::kRows] = row_of(cut, i % C::kRows);
    // Slot 0: the item began in an earlier CTA.
    if (i % C::kRows == 0)
      run.slot = cut.first >= cta_r0 && cut.first + cut.units <= cta_r1 ? -1 : (cut.first >= cta_r0 ? 1 : 0);
  }
  __syncthreads();
  // An output of four columns a thread, four of them at a time: the heads among their parts (in
  // L2) are asked for together.
  constexpr int kOuts = C::kRows * (D / 4), kTogether = 4;
#pragma unroll 1
  for (int i0 = tid; i0 < sh.runs * kOuts; i0 += kTogether * kThreads) {
    float hm[kTogether], hl[kTogether];
    float4 hv[kTogether];
#pragma unroll
    for (int x = 0; x < kTogether; ++x) {
      const int i = i0 + x * kThreads, at = i % kOuts, row = at / (D / 4), c = at % (D / 4) * 4;
      const int eh = i < sh.runs * kOuts ? sh.run[i / kOuts].head : -1;
      hm[x] = -INFINITY;
      hl[x] = 0.f;
      hv[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (eh >= 0) {  // either memory; stores of this CTA's own warps, ordered by its barrier
        const float* q = head_part(eh);
        hm[x] = q[C::kTop + row];
        hl[x] = q[C::kSum + row];
        hv[x] = *reinterpret_cast<const float4*>(q + row * C::kPitch + c);
      }
    }
#pragma unroll
    for (int x = 0; x < kTogether; ++x) {
      const int i = i0 + x * kThreads, at = i % kOuts, row = at / (D / 4), c = at % (D / 4) * 4;
      if (i >= sh.runs * kOuts) break;
      const int64_t to = sh.row_at[i / kOuts][row];
      if (to < 0) continue;
      const auto run = sh.run[i / kOuts];
      Sum s;
      s.m = hm[x];
      s.l = hl[x];
      s.v = hv[x];
      constexpr int kTails = 4;
#pragma unroll 1
      for (int v = run.first >= 0 ? run.first : kWarps; v <= run.last; v += kTails) {
        float mk[kTails], lk[kTails];
        float4 f[kTails];
#pragma unroll
        for (int y = 0; y < kTails; ++y) {
          const int w = min(v + y, static_cast<int>(run.last));
          const float* q = tail_part(w);
          const bool have = v + y <= run.last && sh.has_tail[w];  // warps without a unit have none: no weight
          const float4 z = *reinterpret_cast<const float4*>(q + row * C::kPitch + c);
          mk[y] = have ? q[C::kTop + row] : -INFINITY;
          lk[y] = have ? q[C::kSum + row] : 0.f;
          f[y] = have ? z : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        s.add(mk, lk, f);
      }
      if (run.slot < 0) {
        *reinterpret_cast<uint2*>(p.O + to + c) = s.value();
      } else {
        float* out = cta_parts + (2 * static_cast<int64_t>(blockIdx.x) + run.slot) * C::kPart;
        __stcg(reinterpret_cast<float4*>(out + row * C::kPitch + c), s.v);
        if (c == 0) {
          __stcg(out + C::kTop + row, s.m);
          __stcg(out + C::kSum + row, s.l);
        }
      }
    }
  }
  __syncthreads();  // before the tickets: their release covers the CTA's stores
  // Only the first and the last run can be of an item of other CTAs too.
  constexpr int kAtOnce = NT == 1 ? 1 : 4, kBatch = NT == 1 ? 8 : 4;
  // An item whose parts would take the threads more turns than this is joined in two steps (one
  // sequence of 32768, 16 queries of one head: 20.9 us, in one step of 38 turns 47.8; 4 items of
  // 16768 keys, 32 queries, 10 turns: 35.4 and 57.6; 7 queries, 2 turns: 11.0 and 9.9).
  constexpr int kTurns = 4;
  uint32_t* counters = static_cast<uint32_t*>(p.ws);
  // The parts of a step of an item's join are places lo .. hi - 1 from base on, the item's first
  // in the odd half of its place, all others in the even ones.
  struct Step {
    uint32_t base, lo, hi, first;
    uint32_t counter, sum;  // the step's counter; the part that its sum is, unless it is the last
    bool ends;
  };
  auto cut_of = [&](int r) { return sh.run[r].first >= 0 ? sh.tail[sh.run[r].first] : sh.head[sh.run[r].head]; };
  auto outs_of = [&](const Cut& cut) {  // of the rows that the item has
    return min(C::kRows, rows_all - cut.item % qblocks * C::kRows) * (D / 4);
  };
  // Step `pass` of the join of a run's item.
  auto step_of = [&](int r, int pass) {
    const Cut cut = cut_of(r);
    const uint32_t k0 = split.worker(cut.first), k1 = split.worker(cut.first + cut.units - 1), team = k0 / kTeam;
    const uint32_t at = (blockIdx.x - k0) / kTeam, from = k0 + at * kTeam;
    if (pass > 0) return Step{2 * kMaxCtas, team, team + (k1 - k0) / kTeam + 1, team, k0, 0, true};
    if (k1 - k0 < kTurns * kBatch * max(kThreads / outs_of(cut), 1)) return Step{0, k0, k1 + 1, k0, k0, 0, true};
    const uint32_t place = 2 * (team + at) + (at == 0);
    return Step{0, from, min(from + kTeam, k1 + 1), k0, kMaxCtas + place, 2 * kMaxCtas + place, false};
  };
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    // A CTA is the first one of at most one item that goes on after it: that item's counter is
    // the first CTA's.  (The barrier before orders the CTA's stores; the ticket's release covers
    // them.)
    if (tid == 0 || tid == 32) {
      const int side = tid == 0 ? 0 : 1, r = pass > 0 ? sh.last[side] : side == 0 ? 0 : sh.runs - 1;
      int last = -1;
      if (pass > 0 ? r >= 0 && !sh.ends[side] : r >= side && r < sh.runs && sh.run[r].slot >= 0) {
        const Step step = step_of(r, pass);
        if (take_ticket(counters + step.counter) == step.hi - step.lo - 1) {
          counters[step.counter] = 0;  // every contributor has its ticket: ready for the next call
          last = r;
          sh.ends[side] = step.ends;
        }
      }
      sh.last[side] = last;
    }
    __syncthreads();
    if (sh.last[0] < 0 && sh.last[1] < 0) return;

    // ---- the steps whose last part was this CTA's.  The outputs of both are one row of outputs
    // of four columns; a thread takes kAtOnce of them, and asks for kBatch parts of each
    // together.  Many parts of few outputs: groups of threads take the parts in turn, and join
    // through shared memory.
    Step step[2];
    uint32_t most = 0;
    int outs[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int last = sh.last[side];
      outs[side] = 0;
      step[side] = Step{0, 0, 0, 0, 0, 0, true};
      if (last < 0) continue;
      step[side] = step_of(last, pass);
      outs[side] = outs_of(cut_of(last));
      most = max(most, step[side].hi - step[side].lo);
    }
    const int n = outs[0] + outs[1];
    const int groups = most > kBatch && 2 * n <= kThreads ? kThreads / n : 1;
    float* mid = reinterpret_cast<float*>(smem);  // [thread][6]
    auto emit = [&](const Sum& s, bool second, int at) {
      const int row = at / (D / 4), c = at % (D / 4) * 4;
      if (second ? step[1].ends : step[0].ends) {
        *reinterpret_cast<uint2*>(p.O + sh.row_at[sh.last[second]][row] + c) = s.value();
        return;
      }
      float* out = cta_parts + static_cast<int64_t>(second ? step[1].sum : step[0].sum) * C::kPart;
      __stcg(reinterpret_cast<float4*>(out + row * C::kPitch + c), s.v);
      if (c == 0) {
        __stcg(out + C::kTop + row, s.m);
        __stcg(out + C::kSum + row, s.l);
      }
    };
#pragma unroll 1
    for (int i0 = tid; i0 < groups * n; i0 += kAtOnce * kThreads) {
      Sum s[kAtOnce];
      int at[kAtOnce], row[kAtOnce];
      bool second[kAtOnce];
      uint32_t k[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int i = i0 + x * kThreads, grp = groups > 1 ? i / n : 0, o = i - grp * n;
        second[x] = o >= outs[0];
        at[x] = i < groups * n ? o - (second[x] ? outs[0] : 0) : -1;
        row[x] = at[x] >= 0 ? at[x] / (D / 4) : 0;
        k[x] = (second[x] ? step[1].lo : step[0].lo) + grp;
      }
#pragma unroll 1
      for (uint32_t done = 0; done < most; done += kBatch * groups) {
        float mk[kAtOnce][kBatch], lk[kAtOnce][kBatch];
        float4 v[kAtOnce][kBatch];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x)
#pragma unroll
          for (int y = 0; y < kBatch; ++y) {
            const uint32_t kk = k[x] + done + y * groups;
            const Step& st = second[x] ? step[1] : step[0];
            const float* q = cta_parts + static_cast<int64_t>(st.base + 2 * kk + (kk == st.first)) * C::kPart;
            const bool in = at[x] >= 0 && kk < st.hi;
            mk[x][y] = in ? __ldcg(q + C::kTop + row[x]) : -INFINITY;
            lk[x][y] = in ? __ldcg(q + C::kSum + row[x]) : 0.f;
            v[x][y] = in ? __ldcg(reinterpret_cast<const float4*>(q + row[x] * C::kPitch + at[x] % (D / 4) * 4))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) s[x].add(mk[x], lk[x], v[x]);
      }
      if (groups == 1) {
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x)
          if (at[x] >= 0) emit(s[x], second[x], at[x]);
      } else {  // (one turn)
        float* d = mid + tid * 6;
        d[0] = s[0].m;
        d[1] = s[0].l;
        d[2] = s[0].v.x;
        d[3] = s[0].v.y;
        d[4] = s[0].v.z;
        d[5] = s[0].v.w;
      }
    }
    if (groups > 1) {  // uniform over the CTA
      __syncthreads();
      if (tid < n) {
        Sum s;
#pragma unroll 4
        for (int x = 0; x < groups; ++x) {
          const float* d = mid + (x * n + tid) * 6;
          const float mk[1] = {d[0]}, lk[1] = {d[1]};
          const float4 v[1] = {make_float4(d[2], d[3], d[4], d[5])};
          s.add(mk, lk, v);
        }
        const bool second = tid >= outs[0];
        emit(s, second, tid - (second ? outs[0] : 0));
      }
    }
    if (step[0].ends && step[1].ends) return;
    __syncthreads();
  }
}

template <int D, int NT, bool TREE>
cudaError_t launch_variant(const Kv4AttnParams& p, int sms, cudaStream_t s) {
  using C = Cfg<D, NT>;
  auto kern = kv4_attention_kernel<D, NT, TREE>;
  static std::atomic<uint64_t> attr_done{0};
  const cudaError_t e = ensure_smem_attr(kern, C::kSmem, attr_done);
  if (e != cudaSuccess) return e;
  const int rows = static_cast<int>(p.Lq) * p.group;
  Kv4AttnParams q = p;
  q.one_copy = p.page_size % C::kUnit == 0;
  q.fault = g_fault_injection;
  return launch_pdl(kern, dim3(static_cast<unsigned>(sms < kMaxCtas ? sms : kMaxCtas)), dim3(C::kThreads), C::kSmem,
                    s, q, (rows + C::kRows - 1) / C::kRows);
}

// Query rows of a block: the fewest tiles of 8 that hold them, at most 4.
int tiles_of(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

template <int D, int NT>
constexpr int64_t ws_bytes() {
  using C = Cfg<D, NT>;
  return kCounterBytes + (static_cast<int64_t>(kMaxCtas) * (C::kWarps + 2) + kTeams) * C::kPart * 4;
}

}  // namespace

int64_t kv4_attention_ws_bytes(int64_t Lq, int64_t heads_q, int64_t heads_kv, int d) {
  const int nt = tiles_of(Lq * (heads_q / heads_kv));
  const int64_t rows = d == 128 ? (nt == 1 ? ws_bytes<128, 1>() : nt == 2 ? ws_bytes<128, 2>() : ws_bytes<128, 4>())
                                : (nt == 1 ? ws_bytes<64, 1>() : nt == 2 ? ws_bytes<64, 2>() : ws_bytes<64, 4>());
  // Trees of more than 16 rows take the other kernel, which has parts of its own.
  const int64_t tree = nt == 4 ? kv4_tree_ws_bytes(d) : 0;
  return rows > tree ? rows : tree;
}

template <int D, bool TREE>
cudaError_t launch_rows_d(const Kv4AttnParams& p, int sms, cudaStream_t s) {
  const int nt = tiles_of(p.Lq * p.group);
  if (nt == 1) return launch_variant<D, 1, TREE>(p, sms, s);
  if constexpr (!TREE)  // (trees of more than 16 rows do not come here)
    if (nt == 4) return launch_variant<D, 4, false>(p, sms, s);
  return launch_variant<D, 2, TREE>(p, sms, s);
}

template <bool TREE>
cudaError_t launch_rows(const Kv4AttnParams& p, int d, int sms, cudaStream_t s) {
  return d == 128 ? launch_rows_d<128, TREE>(p, sms, s) : launch_rows_d<64, TREE>(p, sms, s);
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, int d, int sms, cudaStream_t s) {
  if (!p.mask) return launch_rows<false>(p, d, sms, s);
  // Trees of more than 16 query rows a cache head.  8 heads, d = 128,
  // us here and there: one sequence of 8208 tokens 8 rows 14.6 and 18.1, 16 rows 22.5 and 18.2, 32 rows 37.6 and
  // 18.2; 8 of them 16 rows 32.7 and 58.3, 32 rows 56.0 and 58.5; 64 of 600 tokens 16 rows 24.8 and 54.6, 32 rows
  // 47.8 and 55.9.
  if (p.Lq * p.group > 16) return launch_kv4_tree(p, d, sms, s);
  return launch_rows<true>(p, d, sms, s);
}

}  // namespace dg
