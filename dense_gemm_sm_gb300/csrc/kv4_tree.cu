// kv4_tree.cu -- attention of trees of drafted tokens over the paged 4-bit cache, on tcgen05: for more
// than 16 query rows per cache head (fewer take kv4_attention.cu's kernel, whose MMAs are 8 rows wide).
//
// Query i < nodes of a sequence sees the keys before base = len - nodes and those of the newest `nodes`
// that its mask names.  With K_j = kz_j + ks_j kc_j and V_j = vz_j + vs_j vc_j (codes 0..15):
//   score_j = ks_j (q . (16 + kc_j)) + (kz_j - 16 ks_j) sum(q),   p_j = 2^(c score_j - reference),
//   O = [sum_j P_j (16 + vc_j) - 24 sum_j P_j + sum_j p_j (vz_j + 8 vs_j)] / sum_j p_j,  P_j = bf16(p_j vs_j),
// so that codes enter the products exactly (16 + c is a BF16 number, put together by a shift and one
// AND-OR for two codes) and what the rounding of P multiplies is vc_j - 8, V's deviation from the middle
// of its range.  sum_j P_j is a column of ones beside V.
//
// The rows of the group's heads and of all nodes (row = node * group + head) share each expanded key:
// a block of 128 of them is the MMA's M.  Per unit of 128 keys (d = 128) the tensor cores need 1040 cycles,
// the exponentials 1024, expanding K and V 512 of the logic pipe.  Warps:
//   0-15   softmax, four threads a row (32 keys each; they exchange the maximum), epilogue;
//   16-19  expansion: a thread per key writes K's row, then 8 keys of V's columns, as K-major operands
//          (d in the order in which the codes come out of their words, which Q's rows follow; V's
//          pieces hold two tokens of a column side by side, so that V comes out transposed);
//   20     copies of records into a ring;   21  products: S_j+1 before P_j V_j, so that the softmax of
//          one unit overlaps the product of the next.  P_j takes the place of S_j in tensor memory.
// Units of all (sequence, head, block of rows) items are cut evenly over one CTA per SM.  A cut item's parts
// go to the workspace, and a small second kernel joins them in CTA order, spread over all SMs (one
// CTA alone would read 66 kB for each part).
// Measured: 4 sequences of 24064 tokens, 64 nodes, 32 heads over 8, d = 128: 150 us, 1.9 us a unit, of shared memory's wavefronts
// 73 % (most are the four numbers that a key brings, read for each row), of the tensor pipe 30 %.  Eight softmax
// warps of 64 keys 172; sixteen that keep four rows in a thread, so that a key's numbers are read once for 16
// rows, 177 (tcgen05.ld and st of 16 lanes); four more warps that expand V alone 159.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

constexpr int kMaxCtas = 160;    // CTAs that the workspace has room for
constexpr int kKeys = 128, kRows = 128, kUnitRecs = kKeys / kKv4Tokens;
constexpr int kSoftWarps = 16, kExpandWarps = 4;
constexpr int kParts = kSoftWarps / 4, kPartKeys = kKeys / kParts;  // of a unit's keys, one to each warp of a quadrant
constexpr int kFirstExpand = kSoftWarps, kCopier = kFirstExpand + kExpandWarps, kIssuer = kCopier + 1;
constexpr int kThreads = 32 * (kIssuer + 1);
constexpr uint32_t kMinUnits = 1;   // of a CTA (2: one sequence of 512 tokens 14.4 -> 15.2 us)
constexpr float kSlack = 8.f;       // the reference follows the maximum only when that has outgrown it by this
constexpr int64_t kCounterBytes = 1024;  // of kv4_attention.cu's kernel, left as they are
// Tensor memory: S (two buffers; P_j takes the place of S_j), O and the column of sums of P.
constexpr uint32_t kOCol = 256, kTmemCols = 512;

template <int D>
struct Cfg {
  static constexpr int kBoxes = D / 64;                        // of 64 columns of d, 128-byte rows
  static constexpr uint32_t kQBytes = kBoxes * kRows * 128, kKBytes = kBoxes * kKeys * 128;
  static constexpr int kN = D + 16;                            // columns of the second product: V's, ones, 15 zeros
  static constexpr uint32_t kVBox = kN * 128, kVBytes = 2 * kVBox;  // boxes of 64 keys
  static constexpr uint32_t kRec = kv4_record_bytes(D), kRecStride = kRec + 16;  // off multiples of 128 bytes: banks
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kStage = kUnitRecs * kRecStride;
  static constexpr uint32_t kSmem = 1024 + kQBytes + 2 * kKBytes + 2 * kVBytes + kStages * kStage;
  static constexpr int64_t kPart = kRows * D + 2 * kRows;      // floats: [d / 4][row] float4, references, sums
  static_assert(kSmem + 16 * 1024 <= 227 * 1024, "shared memory, with the static part");
};

// A cut item, for the join.
struct Cut {
  int32_t valid, lo, hi, slot;  // CTAs that have parts, the first one's place
  int32_t b, head, row0, live;
};

struct Shared {
  alignas(16) float a[2][kKeys], b[2][kKeys], vs[2][kKeys], vz[2][kKeys];  // of a unit's keys
  uint32_t valid[2][kKeys / 32];
  float top[2][kParts][kRows];                                 // parts' maxima
  float l[kParts][kRows], z[kParts][kRows], q[kParts][kRows];
  alignas(16) int32_t okay[2][4][kParts];
  uint64_t cfull[4], cempty[4], kfull[2], kempty[2], vfull[2], vempty[2], nempty[2], sfull[2], pfull[2], odone[2];
  uint64_t qfull, oread, drain;
  uint32_t stage_mask[4];
  int32_t stage_keys[4], stage_shared[4];  // keys of a stage's unit, keys before the first that not every query sees
  uint32_t tmem_base, abort, verdict, issued, total, item;
  struct Start {
    uint32_t b;
    int32_t item, u, units, blocks, len, nodes;
  } start, at[kSoftWarps];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two FP32 numbers in a 64-bit register, low one first, and the packed operations on them.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ ulonglong2 lds_f4(const float* a) {  // four of them
  return *reinterpret_cast<const ulonglong2*>(a);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t w;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(a));
  return w;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint32_t elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p;
}
// The whole warp comes here, its elected lane issues (as in w4.cu).
template <bool ACCUMULATE>
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(ACCUMULATE ? 1 : 0), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a), "r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_x1(uint32_t a, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld_x1(uint32_t a) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void soft_bar() { asm volatile("bar.sync 1, 512;" ::: "memory"); }
__device__ __forceinline__ void part_bar(int quadrant) { asm volatile("bar.sync %0, 128;" ::"r"(2 + quadrant) : "memory"); }

// Codes -> BF16 pairs 16 + code: bits 3-6 of 0x4180.
struct Magic {
  uint32_t mask, offset;  // in registers: as constants the AND and the OR are two instructions
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x00780078;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(offset));
  }
  template <int N>
  __device__ __forceinline__ uint32_t pair(uint32_t w) const {  // of the halves' N-th nibbles
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(N == 0 ? w << 3 : w >> (4 * N - 3)), "r"(mask), "r"(offset));
    return d;
  }
};

// `units` cut evenly over `workers`, the first `rem` of which have one more.
struct Even {
  uint32_t q, rem;
  __device__ __forceinline__ Even(uint32_t units, uint32_t workers) : q(units / workers), rem(units - q * workers) {}
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return c * q + (c < rem ? c : rem); }
  __device__ __forceinline__ uint32_t worker(uint32_t x) const {  // that has unit x
    const uint32_t long_units = rem * (q + 1);
    return x < long_units ? x / (q + 1) : rem + (x - long_units) / q;
  }
};
// The cut of all units over CTAs.  A CTA that goes from one item to the next pays 2.7 us between them, as
// for nearly two units: items that all have the same number of units (`item`; 0: they do not) get CTAs of their
// own where no share grows by more than one unit by that (16 nodes over 8208 tokens: 8 items of 65 units).
struct Split {
  uint32_t ctas, per, item;  // per: CTAs of an item, 0: cut without regard to items
  Even cut;
  static __device__ __forceinline__ uint32_t ceil(uint32_t a, uint32_t b) { return (a + b - 1) / b; }
  __device__ __forceinline__ Split(uint32_t total, uint32_t item, uint32_t grid)
      : ctas(min(ceil(total, kMinUnits), grid)), per(0), item(item), cut(total, max(ctas, 1u)) {
    if (item == 0 || total == 0) return;
    const uint32_t items = total / item, k = min(grid / items, ceil(item, kMinUnits));
    if (k == 0 || ceil(item, k) > ceil(total, ctas) + 1) return;
    per = k;
    ctas = k * items;
    cut = Even(item, k);
  }
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return per ? c / per * item + cut.start(c % per) : cut.start(c); }
  __device__ __forceinline__ uint32_t worker(uint32_t x) const { return per ? x / item * per + cut.worker(x % item) : cut.worker(x); }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_tree_kernel(const Kv4AttnParams p, Cut* cuts) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base, sK = sQ + C::kQBytes, sV = sK + 2 * C::kKBytes, ring = sV + 2 * C::kVBytes;
  volatile uint32_t* abort = &sh.abort;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&sh.cfull[s]), 1);
      mbar_init(smem_u32(&sh.cempty[s]), kExpandWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.kfull[s]), kExpandWarps);
      mbar_init(smem_u32(&sh.kempty[s]), 1);
      mbar_init(smem_u32(&sh.vfull[s]), kExpandWarps);
      mbar_init(smem_u32(&sh.vempty[s]), 1);
      mbar_init(smem_u32(&sh.nempty[s]), kSoftWarps);
      mbar_init(smem_u32(&sh.sfull[s]), 1);
      mbar_init(smem_u32(&sh.pfull[s]), kSoftWarps);
      mbar_init(smem_u32(&sh.odone[s]), 1);
    }
    mbar_init(smem_u32(&sh.qfull), kSoftWarps);
    mbar_init(smem_u32(&sh.oread), kSoftWarps);
    mbar_init(smem_u32(&sh.drain), 1);
    sh.abort = 0;
    sh.issued = 0;
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  // The columns beside V: ones, zeros.  (All of a 128-byte row, so the swizzle moves nothing.)
  for (int i = tid; i < 2 * 2 * 16 * 8; i += kThreads) {
    const int piece = i & 7, row = i >> 3 & 15, box = i >> 7;
    const uint32_t one = row == 0 ? 0x3F803F80u : 0u;
    st_shared_v4(sV + box * C::kVBox + (D + row) * 128 + piece * 16, one, one, one, one);
  }
  fence_proxy_async_smem();
  pdl_trigger();
  pdl_wait();

  // ---- sequences: their units, and where this CTA's share begins
  const int32_t cap = static_cast<int32_t>(p.ldt * p.page_size);
  const uint32_t batch = static_cast<uint32_t>(p.batch);
  auto len_of = [&](uint32_t b) -> int32_t { return min(max(p.lens[b], 0), cap); };
  auto nodes_of = [&](uint32_t b) -> int32_t {
    return min(max(p.nodes ? p.nodes[b] : static_cast<int32_t>(p.Lq), 0), static_cast<int32_t>(p.Lq));
  };
  auto key_units = [](int32_t len) { return (len + kKeys - 1) / kKeys; };
  auto row_blocks = [&](int32_t nodes) { return (nodes * p.group + kRows - 1) / kRows; };
  if (warp == 0) {
    // A lane takes a run of sequences, and keeps what it read of the first.
    const uint32_t per = (batch + 31) / 32, b_lo = min(lane * per, batch), b_hi = min(b_lo + per, batch);
    int32_t len0 = 0, nodes0 = 0;
    uint32_t mine = 0, low = ~0u, high = 0;  // units; the fewest and the most of an item
    for (uint32_t b = b_lo; b < b_hi; ++b) {
      const int32_t n = p.lens[b], m = p.nodes ? p.nodes[b] : static_cast<int32_t>(p.Lq);
      if (blockIdx.x == 0 && (n < 0 || n > cap || m < 0 || m > p.Lq)) atomicCAS(p.index_word, 0u, kDevBadIndex);
      const int32_t len = min(max(n, 0), cap), nodes = min(max(m, 0), static_cast<int32_t>(p.Lq));
      if (b == b_lo) len0 = len, nodes0 = nodes;
      const uint32_t n_units = key_units(len) * row_blocks(nodes) * p.heads;
      if (n_units) low = min(low, key_units(len)), high = max(high, key_units(len));
      mine += n_units;
    }
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t total = __shfl_sync(~0u, incl, 31);
    low = __reduce_min_sync(~0u, low);
    high = __reduce_max_sync(~0u, high);
    const uint32_t same = low == high ? high : 0;
    const Split split(total, same, gridDim.x);
    if (lane == 0) sh.total = total, sh.item = same;
    if (blockIdx.x < split.ctas) {
      const uint32_t r = split.start(blockIdx.x);
      const int owner = __ffs(__ballot_sync(~0u, r < incl)) - 1;
      if (lane == owner) {
        uint32_t at = incl - mine, b = b_lo;
        for (;; ++b) {
          const int32_t len = b == b_lo ? len0 : len_of(b), nodes = b == b_lo ? nodes0 : nodes_of(b);
          const int32_t units = key_units(len), blocks = row_blocks(nodes);
          const uint32_t n = units * blocks * p.heads;
          if (r < at + n) {
            const int32_t item = (r - at) / units;
            sh.start = {b, item, static_cast<int32_t>(r - at) - item * units, units, blocks, len, nodes};
            break;
          }
          at += n;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, sh.tmem_base, 0);
  const Split split(sh.total, sh.item, gridDim.x);
  const bool active = blockIdx.x < split.ctas;
  const uint32_t u0 = active ? split.start(blockIdx.x) : 0, n = active ? split.start(blockIdx.x + 1) - u0 : 0;

  // The pieces of items, one after the other.
  Shared::Start at = sh.start;
  auto forward = [&](Shared::Start& at, int32_t k) {  // k units on; there are more units
    at.u += k;
    if (at.u < at.units) return;
    at.u = 0;
    if (++at.item < p.heads * at.blocks) return;
    at.item = 0;
    do {
      ++at.b;
      at.len = len_of(at.b);
      at.nodes = nodes_of(at.b);
      at.units = key_units(at.len);
      at.blocks = row_blocks(at.nodes);
    } while (at.units * at.blocks == 0);
  };

  if (warp == kCopier) {
    // ------------------------------------------------------------ copies: a lane for each record of a unit
    const int32_t page_recs = p.page_size / kKv4Tokens;
    const int64_t head_bytes = static_cast<int64_t>(page_recs) * C::kRec;
    uint32_t s = 0, ph = 1, i = 0;
    int32_t page = -1;
    uint32_t in = 0;
    bool named = false;
    auto look_up = [&]() {
      const uint32_t rec = at.u * kUnitRecs + lane;
      named = lane < kUnitRecs && static_cast<int32_t>(rec * kKv4Tokens) < at.len;
      // Records are whole: the page of record r is r / (page_size / 16), by multiplication.
      const uint32_t pi = p.page_magic ? __umulhi(rec, p.page_magic) : rec;
      in = rec - pi * page_recs;
      page = named ? p.table[static_cast<int64_t>(at.b) * p.ldt + pi] : -1;
    };
    if (n > 0) look_up();
    for (; i < n; ++i) {
      const bool have = page >= 0 && page < p.pages;
      if (named && !have) atomicCAS(p.index_word, 0u, kDevBadIndex);
      const uint32_t mask = __ballot_sync(~0u, have);
      const uint8_t* src = p.data + (static_cast<int64_t>(page) * p.heads + at.item / at.blocks) * head_bytes + static_cast<int64_t>(in) * C::kRec;
      const int32_t keys = min(kKeys, at.len - at.u * kKeys);
      if (!mbar_wait_warp(smem_u32(&sh.cempty[s]), ph, abort, p.status, kDevTimeoutProducer)) break;
      const uint32_t f = smem_u32(&sh.cfull[s]);
      if (lane == 0) {
        sh.stage_mask[s] = mask;
        sh.stage_keys[s] = keys;
        sh.stage_shared[s] = at.len - at.nodes - at.u * kKeys;
        mbar_arrive_expect_tx(f, __popc(mask) * C::kRec);
      }
      __syncwarp();
      if (have) bulk_load(ring + s * C::kStage + lane * C::kRecStride, src, C::kRec, f);
      if (++s == C::kStages) s = 0, ph ^= 1u;
      if (i + 1 < n) {
        forward(at, 1);
        look_up();
      }
    }
    if (lane == 0) sh.issued = i;
    // ---- queries that see nothing
    for (uint32_t b = blockIdx.x; b < batch; b += gridDim.x) {
      const int32_t from = len_of(b) > 0 ? nodes_of(b) : 0, words = p.group * p.heads * (D / 8);  // of 16 bytes, a query
      for (int i = lane; i < (static_cast<int32_t>(p.Lq) - from) * words; i += 32)
        *reinterpret_cast<uint4*>(p.O + b * p.strideO + static_cast<int64_t>(from + i / words) * p.ldo + i % words * 8) = make_uint4(0, 0, 0, 0);
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ products
    constexpr uint32_t idS = idesc_bf16_f32(128, kKeys, false, false), idO = idesc_bf16_f32(128, C::kN, false, false);
    const uint64_t dQ = sdesc_sw128(sQ, 16, 1024), dK = sdesc_sw128(sK, 16, 1024), dV = sdesc_sw128(sV, 16, 1024);
    const uint32_t lead = elect();
    uint32_t qph = 0, oph = 1;
    int32_t left = 0;  // units of the piece that S goes on with
    uint32_t s_rest = n;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return mbar_wait_warp(smem_u32(bar), parity, abort, p.status, kDevTimeoutMma);
    };
    auto scores = [&](uint32_t j) -> bool {
      const uint32_t b = j & 1, ph = (j >> 1) & 1;
      if (left == 0) {
        if (j > 0) forward(at, at.units - at.u);
        left = min(static_cast<uint32_t>(at.units - at.u), s_rest);
        if (!wait(&sh.qfull, qph)) return false;
        qph ^= 1u;
      }
      // (S's place was P's of two units before, whose product comes before this one.)
      if (!wait(&sh.kfull[b], ph)) return false;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * (kRows * 128) + (k & 3) * 32) >> 4;
        if (k == 0) umma_ss<false>(tmem + b * kKeys, dQ + off, dK + b * (C::kKBytes >> 4) + off, idS, lead);
        else umma_ss<true>(tmem + b * kKeys, dQ + off, dK + b * (C::kKBytes >> 4) + off, idS, lead);
      }
      commit(&sh.kempty[b], lead);
      commit(&sh.sfull[b], lead);
      --left;
      --s_rest;
      return true;
    };
    bool ok = n == 0 || scores(0), first = true;
    for (uint32_t j = 0; ok && j < n; ++j) {
      const uint32_t b = j & 1, ph = (j >> 1) & 1;
      const bool last = left == 0;  // of its piece: the next product waits for other queries
      if (!last) ok = scores(j + 1);
      if (!ok || !wait(&sh.vfull[b], ph) || !wait(&sh.pfull[b], ph) || (first && !wait(&sh.oread, oph))) break;
      if (first) oph ^= 1u;
      tc_fence_after();
      const uint64_t v = dV + b * (C::kVBytes >> 4);
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k)
        umma_ts(tmem + kOCol, tmem + b * kKeys + k * 8, v + (((k >> 2) * C::kVBox + (k & 3) * 32) >> 4), idO, !first || k > 0, lead);
      commit(&sh.vempty[b], lead);
      commit(&sh.odone[b], lead);
      first = last;
      if (last && j + 1 < n) ok = scores(j + 1);
    }
    commit(&sh.drain, lead);
    uint32_t never = 0;
    mbar_wait(smem_u32(&sh.drain), 0, &never, p.status, kDevTimeoutDrain);
    __syncwarp();
  } else if (warp >= kFirstExpand) {
    // ------------------------------------------------------------ expansion
    const Magic magic;
    const int t = tid - 32 * kFirstExpand;
    uint32_t s = 0, ph = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return mbar_wait_warp(smem_u32(bar), parity, abort, p.status, kDevTimeoutMma);
    };
    for (uint32_t j = 0; j < n; ++j) {
      const uint32_t b = j & 1, bph = (j >> 1) & 1;
      if (!wait(&sh.cfull[s], ph)) break;
      const uint32_t st = ring + s * C::kStage;
      {
        // K: thread t has key t; 16-byte pieces of its row in an order that keeps banks apart.
        constexpr int kPieces = D / 32;  // of 32 codes
        const int rec = t >> 4, u = t & 15;
        const uint32_t row = st + rec * C::kRecStride + u * (D / 2), r = st + rec * C::kRecStride + 16 * D + u * 4;
        const uint32_t kp = lds32(r), vp = lds32(r + 64);
        const bool valid = ((sh.stage_mask[s] >> rec) & 1u) && t < sh.stage_keys[s], drafted = t >= sh.stage_shared[s];
        if (!wait(&sh.kempty[b], bph ^ 1u)) break;
        const uint32_t out = sK + b * C::kKBytes + t * 128;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const int cc = (c + (D == 128 ? u >> 1 : u >> 2)) & (kPieces - 1);
          const uint4 w = lds128(row + cc * 16);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            st_shared_v4(out + (cc >> 1) * (kKeys * 128) + ((((cc & 1) * 4 + x) ^ (t & 7)) << 4), magic.pair<0>(ws[x]), magic.pair<1>(ws[x]),
                         magic.pair<2>(ws[x]), magic.pair<3>(ws[x]));
        }
        if (!wait(&sh.nempty[b], bph ^ 1u)) break;
        // A slot past the sequence or the cache may hold anything, and so may one of a drafted token, which a query
        // that does not see it weighs by 0: numbers of V that are not finite there become 0, and the score NaN, which
        // the queries that see the key keep and the others replace.
        const float ks = valid ? lo_of(kp) : 0.f, kz = valid ? hi_of(kp) : 0.f, vs = valid ? lo_of(vp) : 0.f, vz = valid ? hi_of(vp) : 0.f;
        const float v8 = fmaf(8.f, vs, vz);
        const bool wild = drafted && !(fabsf(v8) < INFINITY);
        sh.a[b][t] = ks * p.c_log2;
        sh.b[b][t] = wild ? __uint_as_float(0x7FC00000u) : fmaf(-16.f, ks, kz) * p.c_log2;
        sh.vs[b][t] = wild ? 0.f : vs;
        sh.vz[b][t] = wild ? 0.f : v8;
        const uint32_t vote = __ballot_sync(~0u, valid);
        if (lane == 0) sh.valid[b][warp - kFirstExpand] = vote;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.kfull[b]));
      }
      {
        // V: thread t has 8 keys (one half of a record) of d / 8 columns.
        constexpr int kWords = D / 32;  // of four columns, two tokens
        const int octet = t & 15, g = t >> 4;
        const uint32_t src = st + (octet >> 1) * C::kRecStride + 8 * D + (octet & 1) * (4 * D) + g * (D / 2);
        uint32_t w[4][kWords];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if constexpr (D == 128) {
            const uint4 v = lds128(src + x * 16);
            w[x][0] = v.x;
            w[x][1] = v.y;
            w[x][kWords - 2] = v.z;
            w[x][kWords - 1] = v.w;
          } else if (x < 2) {
            const uint4 v = lds128(src + x * 16);
            w[2 * x][0] = v.x;
            w[2 * x][1] = v.y;
            w[2 * x + 1][0] = v.z;
            w[2 * x + 1][1] = v.w;
          }
        }
        if (!wait(&sh.vempty[b], bph ^ 1u)) break;
        const uint32_t out = sV + b * C::kVBytes + (octet >> 3) * C::kVBox + g * (D / 8) * 128;
        auto put = [&](auto nibble, int c) {
          constexpr int N = decltype(nibble)::value;
          const int col = 4 * c + N;  // of the d / 8, a multiple of 8 before them
          st_shared_v4(out + col * 128 + (((octet & 7) ^ (col & 7)) << 4), magic.pair<N>(w[0][c]), magic.pair<N>(w[1][c]),
                       magic.pair<N>(w[2][c]), magic.pair<N>(w[3][c]));
        };
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
          put(std::integral_constant<int, 0>(), c);
          put(std::integral_constant<int, 1>(), c);
          put(std::integral_constant<int, 2>(), c);
          put(std::integral_constant<int, 3>(), c);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.vfull[b]));
          if (p.fault != 1) mbar_arrive(smem_u32(&sh.cempty[s]));
        }
      }
      if (++s == C::kStages) s = 0, ph ^= 1u;
    }
  } else {
    // ------------------------------------------------------------ softmax: a row's keys 32 part .. 32 part + 31
    const int quadrant = warp & 3, part = warp >> 2, row = quadrant * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quadrant * 32) << 16);
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kCounterBytes);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return mbar_wait_warp(smem_u32(bar), parity, abort, p.status, kDevTimeoutEpilogue);
    };
    Shared::Start& at = sh.at[warp];  // (in shared memory, for registers: every lane writes the same)
    at = sh.start;
    float qsum = 0.f;
    // The sum of a row's elements.  An infinite one becomes NaN: codes and zeros may both pull all scores to -Inf,
    // and a row without a score above that is one that sees no key.
    auto sum_of_queries = [&]() {
      const float sum = (sh.q[0][row] + sh.q[1][row]) + (sh.q[2][row] + sh.q[3][row]);
      return fmaf(0.f, sum, sum);
    };
    uint64_t see = 0;  // the row's nodes
    // The piece's queries to shared memory, in the order of K's codes; rows without one are zeros.
    auto load_queries = [&]() {
      const int head = at.item / at.blocks, r = (at.item - head * at.blocks) * kRows + row, i = r / p.group;
      const bool live = i < at.nodes;
      const uint4* src = reinterpret_cast<const uint4*>(p.Q + static_cast<int64_t>(at.b) * p.strideQ + static_cast<int64_t>(i) * p.ldq +
                                                        static_cast<int64_t>(head * p.group + r - i * p.group) * D + part * (D / kParts));
      uint4 w[D / kParts / 8];
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < D / kParts / 8; ++x) w[x] = live ? __ldg(src + x) : make_uint4(0, 0, 0, 0);
      see = live ? __ldg(reinterpret_cast<const unsigned long long*>(p.mask) + static_cast<int64_t>(at.b) * p.Lq + i) : 0;
#pragma unroll
      for (int x = 0; x < D / kParts / 8; ++x) {
        const int piece = part * (D / kParts / 8) + x;
        st_shared_v4(sQ + (piece >> 3) * (kRows * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4), __byte_perm(w[x].x, w[x].z, 0x5410),
                     __byte_perm(w[x].x, w[x].z, 0x7632), __byte_perm(w[x].y, w[x].w, 0x5410), __byte_perm(w[x].y, w[x].w, 0x7632));
        sum += (lo_of(w[x].x) + hi_of(w[x].x)) + (lo_of(w[x].y) + hi_of(w[x].y)) + ((lo_of(w[x].z) + hi_of(w[x].z)) + (lo_of(w[x].w) + hi_of(w[x].w)));
      }
      sh.q[part][row] = sum;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.qfull));
    };
    if (n > 0) load_queries();
    part_bar(quadrant);
    qsum = sum_of_queries();
    int32_t valid_cut = 0;
    uint32_t j = 0;
    while (j < n) {
      const int32_t units = min(static_cast<uint32_t>(at.units - at.u), n - j);
      const int shared0 = at.len - at.nodes - at.u * kKeys - part * kPartKeys;  // keys from the first of this part's that every query sees
      const bool dead = at.item % at.blocks * kRows + quadrant * 32 >= at.nodes * p.group;
      const uint64_t mask = see;
      const uint64_t q2 = f2(qsum, qsum);
      float ref = 0.f, l = 0.f, z = 0.f;
      bool fresh = true;  // no key seen yet: no reference
      bool ok = true;
#pragma unroll 1
      for (int32_t x = 0; x < units; ++x, ++j) {
        const uint32_t b = j & 1, ph = (j >> 1) & 1;
        ok = ok && wait(&sh.sfull[b], ph);  // (what the keys bring was written before their rows of K were taken)
        if (dead) {  // none of the warp's rows is a query's: what P has there reaches no row that is read
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive(smem_u32(&sh.nempty[b]));
            mbar_arrive(smem_u32(&sh.pfull[b]));
          }
          continue;
        }
        uint32_t sv[kPartKeys];
        float top = -INFINITY;
        if (ok) {
          tc_fence_after();
          tmem_ld_32x32b_x32(tl + b * kKeys + part * kPartKeys, sv);
          tmem_ld_wait();
          tc_fence_before();
          // Scores in log2 units, less the reference.
          const uint64_t nref = f2(-ref, -ref);
#pragma unroll
          for (int k = 0; k < kPartKeys; k += 4) {
            const ulonglong2 ka = lds_f4(&sh.a[b][part * kPartKeys + k]), kb = lds_f4(&sh.b[b][part * kPartKeys + k]);
            uint32_t* v = &sv[k];
            const uint64_t s0 = f2_fma(f2(__uint_as_float(v[0]), __uint_as_float(v[1])), ka.x, f2_fma(kb.x, q2, nref));
            const uint64_t s1 = f2_fma(f2(__uint_as_float(v[2]), __uint_as_float(v[3])), ka.y, f2_fma(kb.y, q2, nref));
            v[0] = static_cast<uint32_t>(s0);
            v[1] = static_cast<uint32_t>(s0 >> 32);
            v[2] = static_cast<uint32_t>(s1);
            v[3] = static_cast<uint32_t>(s1 >> 32);
          }
          const int shared_keys = shared0 - x * kKeys;  // of this part, visible to every query
          const uint32_t valid = sh.valid[b][part];
          if (valid != ~0u || shared_keys < kPartKeys) {
            uint32_t vis = shared_keys >= 32   ? ~0u
                           : shared_keys >= 0  ? ((1u << shared_keys) - 1) | static_cast<uint32_t>(mask << shared_keys)
                           : shared_keys > -64 ? static_cast<uint32_t>(mask >> -shared_keys)
                                               : 0u;
            vis &= valid;
#pragma unroll
            for (int k = 0; k < kPartKeys; ++k)
              if (!((vis >> k) & 1u)) sv[k] = 0xFF800000u;  // -inf
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kPartKeys; k += 2) m4[(k >> 1) & 3] = max3(m4[(k >> 1) & 3], __uint_as_float(sv[k]), __uint_as_float(sv[k + 1]));
          top = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
        }
        sh.top[b][part][row] = top;
        if (lane == 0) sh.okay[b][quadrant][part] = ok;
        part_bar(quadrant);
        const int4 okay = *reinterpret_cast<const int4*>(sh.okay[b][quadrant]);
        ok = okay.x && okay.y && okay.z && okay.w;
        if (!ok) break;
        top = fmaxf(max3(sh.top[b][0][row], sh.top[b][1][row], sh.top[b][2][row]), sh.top[b][3][row]);
        // The reference moves for a maximum far above it, and to the first key's.
        const float move = top > -INFINITY && (fresh || top > kSlack) ? top : 0.f;
        const bool moves = __any_sync(~0u, move != 0.f);
        const float r = fresh ? 1.f : ex2(-move);  // (the first key's may be far below 0, and there is nothing to scale)
        fresh = fresh && !(top > -INFINITY);
        if (moves) {
          l *= r;
          z *= r;
          ref += move;
#pragma unroll
          for (int k = 0; k < kPartKeys; ++k) sv[k] = __float_as_uint(__uint_as_float(sv[k]) - move);
        }
        // Weights, and P for the second product.
        uint32_t pw[kPartKeys / 2];
        uint64_t l2[2] = {0, 0}, z2[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kPartKeys; k += 4) {
          const ulonglong2 va = lds_f4(&sh.vs[b][part * kPartKeys + k]), vb = lds_f4(&sh.vz[b][part * kPartKeys + k]);
          const uint32_t* v = &sv[k];
          const uint64_t p0 = f2(ex2(__uint_as_float(v[0])), ex2(__uint_as_float(v[1])));
          const uint64_t p1 = f2(ex2(__uint_as_float(v[2])), ex2(__uint_as_float(v[3])));
          l2[0] = f2_add(l2[0], p0);
          l2[1] = f2_add(l2[1], p1);
          z2[0] = f2_fma(p0, vb.x, z2[0]);
          z2[1] = f2_fma(p1, vb.y, z2[1]);
          const uint64_t w0 = f2_mul(p0, va.x), w1 = f2_mul(p1, va.y);
          pw[k >> 1] = pack2(f2_lo(w0), f2_hi(w0));
          pw[(k >> 1) + 1] = pack2(f2_lo(w1), f2_hi(w1));
        }
        l += (f2_lo(l2[0]) + f2_hi(l2[0])) + (f2_lo(l2[1]) + f2_hi(l2[1]));
        z += (f2_lo(z2[0]) + f2_hi(z2[0])) + (f2_lo(z2[1]) + f2_hi(z2[1]));
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.nempty[b]));
        tc_fence_after();
        tmem_st_x16(tl + b * kKeys + part * (kPartKeys / 2), pw);  // (past the barrier all of the quadrant's S is read)
        if (moves && x > 0) {  // this part's columns of O, and the sums of P, once the product of the unit before is done
          if (!wait(&sh.odone[b ^ 1], ((j - 1) >> 1) & 1)) {
            ok = false;
            continue;  // the next barrier tells the others
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / kParts; c += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(tl + kOCol + part * (D / kParts) + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * r);
            tmem_st_x16(tl + kOCol + part * (D / kParts) + c, o);
          }
          if (part == 0) {
            const uint32_t o = tmem_ld_x1(tl + kOCol + D);
            tmem_ld_wait();
            tmem_st_x1(tl + kOCol + D, __float_as_uint(__uint_as_float(o) * r));
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.pfull[b]));
      }
      // ---- the next piece's queries: all of this one's scores are in registers
      const bool more = ok && j < n;
      const Shared::Start now = at;
      const int head = now.item / now.blocks, row0 = (now.item - head * now.blocks) * kRows;
      if (more) {
        Shared::Start next = now;
        forward(next, units);
        __syncwarp();
        at = next;
        __syncwarp();
        load_queries();
      }
      if (ok) ok = wait(&sh.odone[(j - 1) & 1], ((j - 1) >> 1) & 1);
      sh.l[part][row] = l;
      sh.z[part][row] = z;
      // One decision of the warps, so that none is left alone in a barrier.
      if (!ok) *abort = 1;
      soft_bar();
      if (tid == 0) sh.verdict = *abort;
      l = (sh.l[0][row] + sh.l[1][row]) + (sh.l[2][row] + sh.l[3][row]);
      z = (sh.z[0][row] + sh.z[1][row]) + (sh.z[2][row] + sh.z[3][row]);
      qsum = sum_of_queries();
      soft_bar();
      if (sh.verdict) break;
      tc_fence_after();
      const uint32_t ps = tmem_ld_x1(tl + kOCol + D);
      tmem_ld_wait();
      const float add = fmaf(-24.f, __uint_as_float(ps), z);
      const bool whole = units == now.units;
      const int r = row0 + row, i = r / p.group;
      const bool live = i < now.nodes;
      uint16_t* out = p.O + static_cast<int64_t>(now.b) * p.strideO + static_cast<int64_t>(i) * p.ldo +
                      static_cast<int64_t>(head * p.group + r - i * p.group) * D + part * (D / kParts);
      const uint32_t first = u0 + (j - units) - now.u;  // the item's first unit
      const int slot = u0 >= first ? 0 : 1;             // of the parts of a CTA: the item that it begins in, or ends in
      float* mine = parts + (2 * static_cast<int64_t>(blockIdx.x) + slot) * C::kPart;
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int c = 0; c < D / kParts; c += 16) {
        uint32_t o[16];
        tmem_ld_32x32b_x16(tl + kOCol + part * (D / kParts) + c, o);
        tmem_ld_wait();
        if (whole) {
          if (live) {
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2((__uint_as_float(o[k + 2 * e]) + add) * inv, (__uint_as_float(o[k + 2 * e + 1]) + add) * inv);
              *reinterpret_cast<uint4*>(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        } else {
          float4* to = reinterpret_cast<float4*>(mine) + (part * (D / kParts / 4) + c / 4) * kRows + row;
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            __stcg(to + k / 4 * kRows, make_float4(__uint_as_float(o[k]) + add, __uint_as_float(o[k + 1]) + add, __uint_as_float(o[k + 2]) + add,
                                                   __uint_as_float(o[k + 3]) + add));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.oread));
      if (!whole && part == 0) {
        __stcg(mine + kRows * D + row, fresh ? -INFINITY : ref);
        __stcg(mine + kRows * D + kRows + row, l);
      }
      if (!whole && now.u == 0 && tid == 0) {  // this CTA is the first of at most one item that goes on after it
        valid_cut = 1;
        cuts[blockIdx.x] = {1, static_cast<int32_t>(blockIdx.x), static_cast<int32_t>(split.worker(first + now.units - 1)), slot,
                            static_cast<int32_t>(now.b), head, row0, min(now.nodes * p.group - row0, kRows)};
      }
    }
    if (tid == 0 && !valid_cut) cuts[blockIdx.x].valid = 0;
  }

  tc_fence_before();
  __syncthreads();
  if (sh.abort && warp == kCopier && lane == 0) {
    // Some wait ran out: the copies in flight land before the CTA ends.
    const uint32_t issued = sh.issued;
    uint32_t never = 0;
    for (uint32_t i = issued > C::kStages ? issued - C::kStages : 0u; i < issued; ++i)
      mbar_wait(smem_u32(&sh.cfull[i % C::kStages]), (i / C::kStages) & 1u, &never, p.status, kDevTimeoutDrain);
  }
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the items that were cut, in CTA order.  Pieces of some columns of all cut items,
// which a block finds by a vote over the other kernel's CTAs, go to the blocks in turn.  Few items have
// many parts each (one sequence in 8 cache heads 19, up to 152): four threads of a block share the parts of a row's
// four columns (one of 8208 tokens, 16 nodes: 27.6 -> 20.8 us).  Many items have few: the four threads
// take four columns each.  A thread has the loads of six parts in flight.
constexpr int kJoinShare = 4, kJoinThreads = kJoinShare * kRows;
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 2) kv4_tree_join_kernel(const Kv4AttnParams p, const Cut* cuts, int ctas) {
  using C = Cfg<D>;
  __shared__ uint32_t votes[kMaxCtas / 32];
  __shared__ float tops[kJoinShare][kRows], sums[kJoinShare][kRows];
  __shared__ float4 values[kJoinShare][kRows];
  static_assert(kMaxCtas % 32 == 0 && kMaxCtas <= kJoinThreads, "a thread for each CTA");
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  if (tid < kMaxCtas) {
    const uint32_t vote = __ballot_sync(~0u, tid < ctas && __ldcg(&cuts[tid].valid) != 0);
    if ((tid & 31) == 0) votes[tid >> 5] = vote;
  }
  __syncthreads();
  int items = 0;
#pragma unroll
  for (int w = 0; w < kMaxCtas / 32; ++w) items += __popc(votes[w]);
  const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.ws) + kCounterBytes);
  const int row = tid % kRows, share = tid / kRows;
  const bool shared = items * (D / 4) <= static_cast<int>(gridDim.x);  // (all at once)
  const int pieces = shared ? D / 4 : D / 4 / kJoinShare, step = shared ? kJoinShare : 1;
#pragma unroll 1
  for (int t = blockIdx.x; t < items * pieces; t += gridDim.x) {
    int nth = t / pieces, from = 0;
    const int col = shared ? t % pieces : t % pieces * kJoinShare + share;  // float4
    while (nth >= __popc(votes[from])) nth -= __popc(votes[from++]);
    const Cut cut = cuts[32 * from + __fns(votes[from], 0, nth + 1)];
    constexpr int kAtOnce = 6;
    float top = -INFINITY, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < cut.live) {
#pragma unroll 1
      for (int k = cut.lo + (shared ? share : 0); k <= cut.hi; k += step * kAtOnce) {
        float m[kAtOnce], n[kAtOnce];
        float4 f[kAtOnce];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          const int at = k + x * step;
          const bool has = at <= cut.hi;
          const float* q = parts + (2 * static_cast<int64_t>(at) + (at == cut.lo ? cut.slot : 0)) * C::kPart;
          m[x] = has ? __ldcg(q + kRows * D + row) : -INFINITY;
          n[x] = has ? __ldcg(q + kRows * D + kRows + row) : 0.f;
          f[x] = has ? __ldcg(reinterpret_cast<const float4*>(q) + col * kRows + row) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float high = top;
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) high = fmaxf(high, m[x]);
        const float ref = high > -INFINITY ? high : 0.f, w0 = ex2(top - ref);
        top = high;
        l *= w0;
        v = make_float4(v.x * w0, v.y * w0, v.z * w0, v.w * w0);
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          if (k + x * step > cut.hi) break;
          const float w = ex2(m[x] - ref);
          l = fmaf(w, n[x], l);
          v = make_float4(fmaf(w, f[x].x, v.x), fmaf(w, f[x].y, v.y), fmaf(w, f[x].z, v.z), fmaf(w, f[x].w, v.w));
        }
      }
    }
    if (shared) {
      tops[share][row] = top;
      sums[share][row] = l;
      values[share][row] = v;
      __syncthreads();
      top = fmaxf(fmaxf(tops[0][row], tops[1][row]), fmaxf(tops[2][row], tops[3][row]));
      const float ref = top > -INFINITY ? top : 0.f;
      l = 0.f;
      v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kJoinShare; ++x) {
        const float w = ex2(tops[x][row] - ref);
        const float4 f = values[x][row];
        l = fmaf(w, sums[x][row], l);
        v = make_float4(fmaf(w, f.x, v.x), fmaf(w, f.y, v.y), fmaf(w, f.z, v.z), fmaf(w, f.w, v.w));
      }
      __syncthreads();
    }
    if ((shared && share) || row >= cut.live) continue;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int r = cut.row0 + row, i = r / p.group;
    uint16_t* out = p.O + static_cast<int64_t>(cut.b) * p.strideO + static_cast<int64_t>(i) * p.ldo +
                    static_cast<int64_t>(cut.head * p.group + r - i * p.group) * D + col * 4;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
  }
}

template <int D>
cudaError_t launch_d(const Kv4AttnParams& p, int sms, cudaStream_t s) {
  using C = Cfg<D>;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = ensure_smem_attr(kv4_tree_kernel<D>, C::kSmem, attr_done);
  if (e != cudaSuccess) return e;
  Kv4AttnParams q = p;
  q.fault = g_fault_injection;
  Cut* cuts = reinterpret_cast<Cut*>(static_cast<uint8_t*>(p.ws) + kCounterBytes + 2 * kMaxCtas * C::kPart * 4);
  const unsigned ctas = static_cast<unsigned>(sms < kMaxCtas ? sms : kMaxCtas);
  e = launch_pdl(kv4_tree_kernel<D>, dim3(ctas), dim3(kThreads), C::kSmem, s, q, cuts);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_tree_join_kernel<D>, dim3(2 * ctas), dim3(kJoinThreads), 0, s, q, static_cast<const Cut*>(cuts), static_cast<int>(ctas));
}

}  // namespace

int64_t kv4_tree_ws_bytes(int d) {
  return kCounterBytes + 2 * kMaxCtas * (d == 128 ? Cfg<128>::kPart : Cfg<64>::kPart) * 4 + kMaxCtas * static_cast<int64_t>(sizeof(Cut));
}

cudaError_t launch_kv4_tree(const Kv4AttnParams& p, int d, int sms, cudaStream_t s) {
  return d == 128 ? launch_d<128>(p, sms, s) : launch_d<64>(p, sms, s);
}

}  // namespace dg
