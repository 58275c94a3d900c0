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
//       O = sum_j P_j (128 + vc_j) + sum_j (p_j vz_j - 128 P_j),   P_j = bf16(p_j vs_j),
//     where the last sum takes the rounded P_j, so the offsets cancel to FP32 rounding.
//   * the order of d in the first product and of keys in the second is free: K rows are read
//     as they lie (a lane 16 bytes, two key rows), V's codes lie in the cache in fragment order.
//   * P goes from the first product's output layout to the second's operand layout by
//     movmatrix, in registers.
// Work: 64-key units of all (sequence, cache head, query block) items, in one row, cut evenly
// over one CTA per SM whatever the lengths; the eight warps of a CTA take its units in turn,
// each with its own ring of bulk copies (one per 16-token record, so pages of any multiple of
// 16 do).  At the end of an item's piece the warps join their maxima, sums and outputs through
// shared memory; an item cut between CTAs is joined, in CTA order, by the last of them to
// arrive (so results do not depend on arrival).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 64;       // keys of a unit
constexpr int kRecs = kUnit / kKv4Tokens;
constexpr int kMaxCtas = 160;   // CTAs that the workspace has room for
constexpr int kMaxRows = 32;    // query rows of a block
// A CTA is given at least this many units, so that small calls use fewer CTAs and joins.
constexpr int kMinUnits = 4;
constexpr int64_t kPartFloats = kMaxRows * (128 + 2);
constexpr int64_t kPartBytes = 2 * kMaxCtas * kPartFloats * 4;  // counters follow at this offset

template <int D, int NT>
struct Cfg {
  static constexpr int kRec = kv4_record_bytes(D);
  static constexpr int kUnitBytes = kRecs * kRec;
  static constexpr int kStages = D == 64 ? 4 : (NT == 4 ? 2 : 3);
  static constexpr int kRing = kWarps * kStages * kUnitBytes;
  static constexpr int kRows = 8 * NT;
  static constexpr int kJoin = kWarps * 8 * 64 * 4;             // one slice: 8 rows x 64 columns per warp
  static constexpr int kQ = NT == 4 ? NT * (D / 16) * 32 * 8 : 0;  // Q fragments (registers otherwise)
  static constexpr int kSmem = kRing + kJoin + kQ;
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

// Codes n of the pair of halves' n-th nibbles -> BF16 pair 128 + code.
template <int N>
__device__ __forceinline__ uint32_t expand(uint32_t w) {
  return ((w >> (4 * N)) & 0x000F000Fu) | 0x43004300u;
}

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

struct Shared {
  uint64_t full[kWarps * 4];
  uint32_t mask[kWarps * 4];   // records of the stage that were copied
  float m[kWarps][kMaxRows], l[kWarps][kMaxRows], z[kWarps][kMaxRows];
  int64_t scan[kThreads / 32];
  int64_t start_b, start_off;
  uint32_t abort, last;
};

__device__ __forceinline__ int64_t start_of(int64_t c, int64_t units, int64_t ctas) { return c * units / ctas; }
__device__ __forceinline__ int64_t cta_of(int64_t x, int64_t units, int64_t ctas) { return ((x + 1) * ctas - 1) / units; }

// Position in the row of all units: unit r is unit u of item `item` of sequence b.
struct Walk {
  int64_t r;
  int64_t b;
  int32_t len, units, item, u;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) kv4_attention_kernel(const Kv4AttnParams p, const int qblocks) {
  using C = Cfg<D, NT>;
  constexpr int KS = D / 16;       // k steps of the first product
  constexpr int MT = D / 16;       // m tiles of the second
  constexpr int W = D / 32;        // words of a lane's share of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kUnitBytes;
  float* join = reinterpret_cast<float*>(smem + C::kRing);
  const uint32_t qfrag = smem_u32(smem) + C::kRing + C::kJoin;

  if (lane == 0)
    for (int s = 0; s < C::kStages; ++s) mbar_init(smem_u32(&sh.full[warp * 4 + s]), 1);
  if (tid == 0) sh.abort = 0;
  fence_barrier_init();
  pdl_trigger();
  pdl_wait();

  const int64_t cap = p.ldt * p.page_size;
  auto len_of = [&](int64_t b) -> int32_t {
    const int32_t n = p.lens[b];
    return n < 0 ? 0 : (n > cap ? static_cast<int32_t>(cap) : n);
  };
  const int ips = p.heads * qblocks;  // items of a sequence
  const int rows_all = static_cast<int>(p.Lq) * p.group;

  // ---- every CTA adds up the units; a thread takes a run of sequences
  const int64_t per = (p.batch + kThreads - 1) / kThreads;
  const int64_t b_lo = tid * per, b_hi = b_lo + per < p.batch ? b_lo + per : p.batch;
  int64_t mine = 0;
  for (int64_t b = b_lo; b < b_hi; ++b) {
    const int32_t n = p.lens[b];
    if (blockIdx.x == 0 && (n < 0 || n > cap)) atomicCAS(p.index_word, 0u, kDevBadIndex);
    mine += (len_of(b) + kUnit - 1) / kUnit;
  }
  mine *= ips;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh.scan[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  incl += before;

  // ---- sequences without a token
  for (int64_t b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (len_of(b) > 0) continue;
    const int64_t n = p.Lq * p.group * p.heads * (D / 8);  // 16-byte words
    for (int64_t i = tid; i < n; i += kThreads) {
      const int64_t row = i / (p.group * p.heads * (D / 8)), c = i % (p.group * p.heads * (D / 8));
      *reinterpret_cast<uint4*>(p.O + b * p.strideO + row * p.ldo + c * 8) = make_uint4(0, 0, 0, 0);
    }
  }
  int64_t ctas = (total + kMinUnits - 1) / kMinUnits;
  if (ctas > gridDim.x) ctas = gridDim.x;
  if (blockIdx.x >= ctas) return;  // whole CTAs
  const int64_t r0 = start_of(blockIdx.x, total, ctas), r1 = start_of(blockIdx.x + 1, total, ctas);

  if (r0 >= incl - mine && r0 < incl) {
    int64_t at = incl - mine, b = b_lo;
    for (;; ++b) {
      const int64_t n = static_cast<int64_t>((len_of(b) + kUnit - 1) / kUnit) * ips;
      if (r0 < at + n) break;
      at += n;
    }
    sh.start_b = b;
    sh.start_off = r0 - at;
  }
  __syncthreads();
  Walk seg;
  seg.r = r0;
  seg.b = sh.start_b;
  seg.len = len_of(seg.b);
  seg.units = (seg.len + kUnit - 1) / kUnit;
  seg.item = static_cast<int32_t>(sh.start_off / seg.units);
  seg.u = static_cast<int32_t>(sh.start_off - static_cast<int64_t>(seg.item) * seg.units);

  auto move_to = [&](Walk& w, int64_t r) {  // r < r1
    int64_t d = r - w.r;
    w.r = r;
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
    w.u += static_cast<int32_t>(d);
  };

  // ---- this warp's copies: units r0 + warp, + 8, ...; the page of the next one is asked for
  // ahead of its turn
  Walk ahead = seg;
  bool more = r0 + warp < r1;
  int nrec = 0, rec_in = 0;
  int32_t page = -1;
  auto prepare = [&]() {
    const int key0 = ahead.u * kUnit;
    nrec = (ahead.len - key0 + kKv4Tokens - 1) / kKv4Tokens;
    nrec = nrec < kRecs ? nrec : kRecs;
    if (lane < nrec) {
      const uint32_t k = key0 + kKv4Tokens * lane, pi = k / static_cast<uint32_t>(p.page_size);
      rec_in = static_cast<int>(k - pi * p.page_size) / kKv4Tokens;
      page = p.table[ahead.b * p.ldt + pi];
    }
  };
  if (more) {
    move_to(ahead, r0 + warp);
    prepare();
  }
  uint32_t put = 0, got = 0;  // units asked for, units used
  auto issue = [&]() {
    const uint32_t s = put % C::kStages;
    const uint32_t bar = smem_u32(&sh.full[warp * 4 + s]);
    const bool in = lane < nrec, ok = in && page >= 0 && page < p.pages;
    if (in && !ok) atomicCAS(p.index_word, 0u, kDevBadIndex);
    const uint32_t mask = __ballot_sync(~0u, ok);
    if (lane == 0) {
      sh.mask[warp * 4 + s] = mask;
      mbar_arrive_expect_tx(bar, __popc(mask) * C::kRec);
    }
    __syncwarp();
    if (ok) {
      const uint8_t* src = p.data + ((static_cast<int64_t>(page) * p.heads + ahead.item / qblocks) *
                                         (p.page_size / kKv4Tokens) + rec_in) * C::kRec;
      bulk_load(ring + s * C::kUnitBytes + lane * C::kRec, src, C::kRec, bar);
    }
    ++put;
    more = ahead.r + kWarps < r1;
    if (more) {
      move_to(ahead, ahead.r + kWarps);
      prepare();
    }
  };
  for (int s = 0; s < C::kStages; ++s)
    if (more) issue();

  // ---- segments: this CTA's piece of one item after the other
  for (;;) {
    const int64_t left = r1 - seg.r;
    const int32_t n = seg.units - seg.u < left ? seg.units - seg.u : static_cast<int32_t>(left);
    const int head = seg.item / qblocks;
    const int row0 = (seg.item - head * qblocks) * C::kRows;
    const uint16_t* qbase = p.Q + seg.b * p.strideQ + static_cast<int64_t>(head) * p.group * D;

    // Q fragments: lane (g, t) takes query row g's elements [t d/4, + d/4).
    uint32_t qf[NT <= 2 ? NT : 1][KS][2];
    float qsum[NT][2];
    int lim[NT][2];  // last key that a column's query sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + nt * 8 + g;
      uint4 w[W];
#pragma unroll
      for (int j = 0; j < W; ++j) w[j] = make_uint4(0, 0, 0, 0);
      if (row < rows_all) {
        const uint4* src = reinterpret_cast<const uint4*>(qbase + static_cast<int64_t>(row / p.group) * p.ldq +
                                                          (row % p.group) * D + t * (D / 4));
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = __ldg(src + j);
      }
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        uint32_t f[4] = {__byte_perm(w[j].x, w[j].z, 0x5410), __byte_perm(w[j].x, w[j].z, 0x7632),
                         __byte_perm(w[j].y, w[j].w, 0x5410), __byte_perm(w[j].y, w[j].w, 0x7632)};
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += lo_of(f[i]) + hi_of(f[i]);
        if constexpr (NT <= 2) {
          qf[nt][2 * j][0] = f[0];
          qf[nt][2 * j][1] = f[1];
          qf[nt][2 * j + 1][0] = f[2];
          qf[nt][2 * j + 1][1] = f[3];
        } else if (warp == nt) {
          // One warp writes each tile; read by all after the barrier below.
          const uint32_t a = qfrag + ((nt * KS + 2 * j) * 32 + lane) * 8;
          asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a), "r"(f[0]), "r"(f[1]) : "memory");
          asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a + 256), "r"(f[2]), "r"(f[3]) : "memory");
        }
      }
      sum += __shfl_xor_sync(~0u, sum, 1);
      sum += __shfl_xor_sync(~0u, sum, 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qsum[nt][e] = __shfl_sync(~0u, sum, (2 * t + e) * 4);
        lim[nt][e] = seg.len - static_cast<int>(p.Lq) + (row0 + nt * 8 + 2 * t + e) / p.group;
      }
    }
    if constexpr (NT == 4) __syncthreads();

    float o[NT][MT][4], m[NT][2], l[NT][2], z[NT][2];
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
      }
    }

    // First unit of this segment that is this warp's.
    const int skip = static_cast<int>((warp - (seg.r - r0)) & (kWarps - 1));
    for (int j = skip; j < n; j += kWarps) {
      const uint32_t s = got % C::kStages, ph = (got / C::kStages) & 1u;
      mbar_wait(smem_u32(&sh.full[warp * 4 + s]), ph, &sh.abort, p.status, kDevTimeoutMma);
      const uint32_t st = ring + s * C::kUnitBytes;
      const uint32_t mask = sh.mask[warp * 4 + s];
      const int key0 = (seg.u + j) * kUnit;

      // ---- S = K Q^T over the unit's 64 keys
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
          const uint32_t a[4] = {expand<0>(ka[w]), expand<1>(ka[w]), expand<2>(ka[w]), expand<3>(ka[w])};
          const uint32_t b[4] = {expand<0>(kb[w]), expand<1>(kb[w]), expand<2>(kb[w]), expand<3>(kb[w])};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t q0, q1;
              if constexpr (NT <= 2) {
                q0 = qf[nt][2 * w + h][0];
                q1 = qf[nt][2 * w + h][1];
              } else {
                asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                             : "=r"(q0), "=r"(q1)
                             : "r"(qfrag + ((nt * KS + 2 * w + h) * 32 + lane) * 8));
              }
              mma_bf16(sc[r][nt], a[2 * h], b[2 * h], a[2 * h + 1], b[2 * h + 1], q0, q1);
            }
        }
      }
      // ---- scores in log2 units, masked where the unit is not all visible
      const bool whole = mask == (1u << kRecs) - 1 && key0 + kUnit <= seg.len - static_cast<int>(p.Lq) + 1;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
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
            if (!whole) {
              const int k = key0 + r * kKv4Tokens + g;
              if (!((mask >> r) & 1u) || k > lim[nt][e]) sc[r][nt][e] = -INFINITY;
              if (!((mask >> r) & 1u) || k + 8 > lim[nt][e]) sc[r][nt][2 + e] = -INFINITY;
            }
            top[nt][e] = fmaxf(top[nt][e], fmaxf(sc[r][nt][e], sc[r][nt][2 + e]));
          }
      }
      // ---- running maximum over the unit (columns' keys lie across the lanes' g)
      float use[NT][2];
      bool grew = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = top[nt][e];
          v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
          v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
          v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
          grew |= v > m[nt][e];
          top[nt][e] = fmaxf(m[nt][e], v);
          use[nt][e] = top[nt][e] > -INFINITY ? top[nt][e] : 0.f;
        }
      if (__any_sync(~0u, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = ex2(m[nt][e] - use[nt][e]);
            l[nt][e] *= f;
            z[nt][e] *= f;
            m[nt][e] = top[nt][e];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[nt][i][e] *= f;
              o[nt][i][2 + e] *= f;
            }
          }
      }
      // ---- P, and O += V^T P^T record by record
#pragma unroll
      for (int r = 0; r < kRecs; ++r) {
        const uint32_t pa = lds1(st + r * C::kRec + 16 * D + 64 + g * 4);
        const uint32_t pb = lds1(st + r * C::kRec + 16 * D + 64 + (g + 8) * 4);
        float s0 = lo_of(pa), z0 = hi_of(pa), s1 = lo_of(pb), z1 = hi_of(pb);
        if (!whole) {  // a row that no query sees may hold anything
          const int k = key0 + r * kKv4Tokens + g;
          const bool have = (mask >> r) & 1u;
          if (!have || k >= seg.len) s0 = z0 = 0.f;
          if (!have || k + 8 >= seg.len) s1 = z1 = 0.f;
        }
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = ex2(sc[r][nt][e] - use[nt][e & 1]);
          const uint32_t x0 = pack2(w[0] * s0, w[1] * s0), x1 = pack2(w[2] * s1, w[3] * s1);
          l[nt][0] += w[0] + w[2];
          l[nt][1] += w[1] + w[3];
          z[nt][0] = fmaf(-128.f, lo_of(x0) + lo_of(x1), fmaf(w[0], z0, fmaf(w[2], z1, z[nt][0])));
          z[nt][1] = fmaf(-128.f, hi_of(x0) + hi_of(x1), fmaf(w[1], z0, fmaf(w[3], z1, z[nt][1])));
          b0[nt] = transpose8x8(x0);
          b1[nt] = transpose8x8(x1);
        }
        uint32_t va[W], vb[W];
        lds(st + r * C::kRec + 8 * D + lane * (D / 8), va);
        lds(st + r * C::kRec + 8 * D + (32 + lane) * (D / 8), vb);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint32_t a[4] = {expand<0>(va[w]), expand<1>(va[w]), expand<2>(va[w]), expand<3>(va[w])};
          const uint32_t b[4] = {expand<0>(vb[w]), expand<1>(vb[w]), expand<2>(vb[w]), expand<3>(vb[w])};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_bf16(o[nt][2 * w + h], a[2 * h], a[2 * h + 1], b[2 * h], b[2 * h + 1], b0[nt], b1[nt]);
        }
      }
      __syncwarp();  // all lanes have read the stage
      ++got;
      if (more) issue();
    }

    // ---- join the warps: maxima and sums first, then the outputs in slices of 8 rows x 64
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], x);
          z[nt][e] += __shfl_xor_sync(~0u, z[nt][e], x);
        }
        if (g == 0) {
          sh.m[warp][nt * 8 + 2 * t + e] = m[nt][e];
          sh.l[warp][nt * 8 + 2 * t + e] = l[nt][e];
        }
      }
    __syncthreads();
    const bool all = seg.u == 0 && n == seg.units;
    const int64_t item0 = seg.r - seg.u;  // the item's first unit
    float* part = static_cast<float*>(p.ws) + (2 * blockIdx.x + (r0 >= item0 ? 0 : 1)) * kPartFloats;
    uint16_t* obase = p.O + seg.b * p.strideO + static_cast<int64_t>(head) * p.group * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nt * 8 + 2 * t + e;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sh.m[w][row]);
        f[e] = m[nt][e] > -INFINITY ? ex2(m[nt][e] - mx) : 0.f;
      }
#pragma unroll
      for (int sl = 0; sl < D / 64; ++sl) {
        // Columns g d/8 + 2 i, + 1 of m tile i: slice sl holds the groups g with g d/8 / 64 == sl.
        if (g / (64 / (D / 8)) == sl) {
          float* dst = join + warp * 512 + (2 * t) * 64 + (g * (D / 8) - sl * 64);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<float2*>(dst + e * 64 + 2 * i) =
                  make_float2((o[nt][i][e] + z[nt][e]) * f[e], (o[nt][i][2 + e] + z[nt][e]) * f[e]);
        }
        __syncthreads();
        const int q = tid >> 5, c = (tid & 31) * 2;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(join + w * 512 + q * 64 + c);
          sum.x += v.x;
          sum.y += v.y;
        }
        const int row = nt * 8 + q;
        if (row0 + row < rows_all) {
          float mx = -INFINITY, tl = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sh.m[w][row]);
#pragma unroll
          for (int w = 0; w < kWarps; ++w)
            tl += sh.m[w][row] > -INFINITY ? sh.l[w][row] * ex2(sh.m[w][row] - mx) : 0.f;
          if (all) {
            const float inv = tl > 0.f ? 1.f / tl : 0.f;
            *reinterpret_cast<uint32_t*>(obase + static_cast<int64_t>((row0 + row) / p.group) * p.ldo +
                                         (row0 + row) % p.group * D + sl * 64 + c) = pack2(sum.x * inv, sum.y * inv);
          } else {
            __stcg(reinterpret_cast<float2*>(part + row * D + sl * 64 + c), sum);
            if (sl == 0 && c == 0) {
              __stcg(part + C::kRows * D + row, mx);
              __stcg(part + C::kRows * D + C::kRows + row, tl);
            }
          }
        }
        __syncthreads();
      }
    }
    if (!all) {
      uint32_t* counter = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.ws) + kPartBytes) + seg.b * ips + seg.item;
      const int64_t c0 = cta_of(item0, total, ctas), c1 = cta_of(item0 + seg.units - 1, total, ctas);
      if (tid == 0) {
        const bool last = take_ticket(counter) == static_cast<uint32_t>(c1 - c0);
        if (last) *counter = 0;  // every contributor has its ticket: ready for the next call
        sh.last = last;
      }
      __syncthreads();
      if (sh.last) {
        const int rows = rows_all - row0 < C::kRows ? rows_all - row0 : C::kRows;
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
          const int row = i / (D / 4), c = (i % (D / 4)) * 4;
          auto part_of = [&](int64_t k) {
            return static_cast<const float*>(p.ws) +
                   (2 * k + (start_of(k, total, ctas) >= item0 ? 0 : 1)) * kPartFloats;
          };
          float mx = -INFINITY;
#pragma unroll 8
          for (int64_t k = c0; k <= c1; ++k) mx = fmaxf(mx, __ldcg(part_of(k) + C::kRows * D + row));
          float tl = 0.f;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int64_t k = c0; k <= c1; ++k) {
            const float* src = part_of(k);
            const float mk = __ldcg(src + C::kRows * D + row), lk = __ldcg(src + C::kRows * D + C::kRows + row);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + row * D + c));
            const float f = mk > -INFINITY ? ex2(mk - mx) : 0.f;
            tl = fmaf(lk, f, tl);
            sum.x = fmaf(v.x, f, sum.x);
            sum.y = fmaf(v.y, f, sum.y);
            sum.z = fmaf(v.z, f, sum.z);
            sum.w = fmaf(v.w, f, sum.w);
          }
          const float inv = tl > 0.f ? 1.f / tl : 0.f;
          *reinterpret_cast<uint2*>(obase + static_cast<int64_t>((row0 + row) / p.group) * p.ldo +
                                    (row0 + row) % p.group * D + c) =
              make_uint2(pack2(sum.x * inv, sum.y * inv), pack2(sum.z * inv, sum.w * inv));
        }
      }
      __syncthreads();  // sh.last is rewritten at the next segment's end
    }
    if (seg.r + n >= r1) break;
    move_to(seg, seg.r + n);
  }
}

template <int D, int NT>
cudaError_t launch_variant(const Kv4AttnParams& p, int sms, cudaStream_t s) {
  auto kern = kv4_attention_kernel<D, NT>;
  static std::atomic<uint64_t> attr_done{0};
  const cudaError_t e = ensure_smem_attr(kern, Cfg<D, NT>::kSmem, attr_done);
  if (e != cudaSuccess) return e;
  const int rows = static_cast<int>(p.Lq) * p.group;
  const int qblocks = (rows + 8 * NT - 1) / (8 * NT);
  return launch_pdl(kern, dim3(static_cast<unsigned>(sms < kMaxCtas ? sms : kMaxCtas)), dim3(kThreads),
                    Cfg<D, NT>::kSmem, s, p, qblocks);
}

// Query rows of a block: the fewest tiles of 8 that hold them, at most 4.
int tiles_of(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

}  // namespace

int64_t kv4_attention_ws_bytes(int64_t batch, int64_t Lq, int64_t heads_q, int64_t heads_kv, int d) {
  (void)d;
  const int64_t rows = Lq * (heads_q / heads_kv), per = 8 * tiles_of(rows);
  return kPartBytes + batch * heads_kv * ((rows + per - 1) / per) * 4;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, int d, int sms, cudaStream_t s) {
  const int nt = tiles_of(p.Lq * p.group);
  if (d == 128)
    return nt == 1 ? launch_variant<128, 1>(p, sms, s) : nt == 2 ? launch_variant<128, 2>(p, sms, s)
                                                                : launch_variant<128, 4>(p, sms, s);
  return nt == 1 ? launch_variant<64, 1>(p, sms, s) : nt == 2 ? launch_variant<64, 2>(p, sms, s)
                                                             : launch_variant<64, 4>(p, sms, s);
}

}  // namespace dg
