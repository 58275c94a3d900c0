// w4.cu -- weights in 4 bits with group scales: quantising them, reading them back, and the
// product of BF16 rows with them.  W is N x K by output column; a group is `group` consecutive k
// of one column n:
//   zero = min w,  scale = bf16((max w - min w) / 15),
//   code = clamp(rne((w - zero) / scale), 0, 15),   w ~ zero + scale * code.
// The minimum of BF16 values is one of them, so zero is exact; the scale is rounded before the
// codes are taken.  Differences, divisions and roundings are IEEE FP32 operations; a constant
// group has scale 0 and codes 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Bit of a word where the code of k % 8 begins: even k in the low half, odd k in the high half.
__device__ __forceinline__ constexpr int code_at(int k) { return 4 * (k >> 1) + 16 * (k & 1); }

// ------------------------------------------------------------------ rows
// HBM-bound: 2 bytes of W, half a byte of codes and 4 / group of parameters an element.  A warp takes 1024 k of
// a row, its four loads together (256 k where those would not fill the GPU's warps twice); a lane holds 8 elements of each, one word of codes, and group / 8
// neighbouring lanes a group.  Neighbouring warps take neighbouring rows, whose parameters lie together.
// Minimum and maximum are reduced as one BF16 pair (maximum, -minimum), quotients come from a reciprocal,
// correctly rounded by one step with their exact remainder, codes are put together from the low bits of
// 1.5 * 2^23 + code.

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// a / b rounded to nearest, for y = 1 / b rounded to nearest: the quotient's approximation a y
// corrected by its remainder, which is exact (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990: right unless all bits of b's significand are set;
// no intermediate result may underflow).
__device__ __forceinline__ float quotient(float a, float b, float y) {
  const float q = a * y;
  return fmaf(fmaf(-q, b, a), y, q);
}

// A warp's piece: row, first word.
struct Piece {
  int64_t n, w;
  __device__ __forceinline__ Piece(int64_t i, int64_t rows, int words) {
    const int64_t block = static_cast<uint64_t>(i) >> 32 || static_cast<uint64_t>(rows) >> 32
                              ? i / rows
                              : static_cast<uint32_t>(i) / static_cast<uint32_t>(rows);
    n = i - block * rows;
    w = block * words;
  }
};

template <int G, bool VEC, int X>
__global__ void __launch_bounds__(kThreads) quantize_w4_kernel(const W4RowsParams p, const int64_t pieces) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < pieces; i += warps) {
    const Piece at(i, p.N, 32 * X);
    const uint16_t* src = p.W + at.n * p.ldw + 8 * (at.w + lane);
    uint32_t* out = reinterpret_cast<uint32_t*>(p.Q + at.n * p.ldq) + at.w + lane;
    uint32_t* prm = p.params + at.n + (8 * (at.w + lane) / G) * p.ldp;
    // Elements from this lane's first word on: 8 or more of them for a whole word, none past the row's end.
    const int64_t rest = p.K - 8 * (at.w + lane);
    uint32_t v[X][4];
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const int64_t left = rest - 256 * x;
      if (VEC && left >= 8) {
        const uint4 q = __ldcs(reinterpret_cast<const uint4*>(src + 256 * x));
        v[x][0] = q.x; v[x][1] = q.y; v[x][2] = q.z; v[x][3] = q.w;
      } else {
        // Past the row's end: its last element again, which changes no range.
        const uint16_t* e = src + 256 * x;
        const int last = left >= 8 ? 7 : static_cast<int>(left) - 1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[x][j] = left <= 0 ? 0u : e[min(2 * j, last)] | static_cast<uint32_t>(e[min(2 * j + 1, last)]) << 16;
      }
    }
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const int64_t left = rest - 256 * x;
      // (maximum, -minimum) of the lane's elements, then of the group; lanes past the end: -inf.
      const uint32_t hi2 = max2(max2(v[x][0], v[x][1]), max2(v[x][2], v[x][3]));
      const uint32_t lo2 = max2(max2(v[x][0] ^ 0x80008000u, v[x][1] ^ 0x80008000u), max2(v[x][2] ^ 0x80008000u, v[x][3] ^ 0x80008000u));
      uint32_t ext = max2(__byte_perm(hi2, lo2, 0x5410), __byte_perm(hi2, lo2, 0x7632));
      if (left <= 0) ext = 0xFF80FF80u;
#pragma unroll
      for (int o = G / 16; o > 0; o >>= 1) ext = max2(ext, __shfl_xor_sync(~0u, ext, o));
      if (left <= 0) continue;
      const float hi = lo_of(ext), lo = __uint_as_float((ext & 0xFFFF0000u) ^ 0x80000000u);
      const float range = __fsub_rn(hi, lo);
      const bool plain = range >= 1e-30f;  // nothing below underflows
      const __nv_bfloat16 sb = __float2bfloat16_rn(plain ? quotient(range, 15.f, 1.f / 15.f) : __fdiv_rn(range, 15.f));
      const float scale = __bfloat162float(sb);
      uint32_t codes = 0;
      if (plain) {
        // A quotient is at most 15 (1 + 2^-8): rounded, at most 15.
        const float inv = __frcp_rn(scale);
        constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, in the low bits
        uint32_t c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float e = k & 1 ? hi_of(v[x][k >> 1]) : lo_of(v[x][k >> 1]);
          c[k] = __float_as_uint(quotient(__fsub_rn(e, lo), scale, inv) + kRound);
        }
        // The low half of a word is the code alone.
        codes = __byte_perm(((c[6] * 16 + c[4]) * 16 + c[2]) * 16 + c[0], ((c[7] * 16 + c[5]) * 16 + c[3]) * 16 + c[1], 0x5410);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float e = k & 1 ? hi_of(v[x][k >> 1]) : lo_of(v[x][k >> 1]);
          const float q = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(e, lo), scale)) : 0.f;
          codes |= static_cast<uint32_t>(fminf(fmaxf(q, 0.f), 15.f)) << code_at(k);
        }
      }
      if (left < 8) {  // codes past K are 0
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k >= left) codes &= ~(15u << code_at(k));
      }
      out[32 * x] = codes;
      if (lane % (G / 8) == 0)
        prm[256 / G * x * p.ldp] = static_cast<uint32_t>(__bfloat16_as_ushort(sb)) | (__float_as_uint(lo) & 0xFFFF0000u);
    }
  }
}

template <int G, bool VEC, int X>
__global__ void __launch_bounds__(kThreads) dequantize_w4_kernel(const W4RowsParams p, const int64_t pieces) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < pieces; i += warps) {
    const Piece at(i, p.N, 32 * X);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.Q + at.n * p.ldq) + at.w + lane;
    const uint32_t* prm = p.params + at.n + (8 * (at.w + lane) / G) * p.ldp;
    uint16_t* out = p.W + at.n * p.ldw + 8 * (at.w + lane);
    const int64_t rest = p.K - 8 * (at.w + lane);
    uint32_t codes[X], words[X];
#pragma unroll
    for (int x = 0; x < X; ++x) {
      if (rest <= 256 * x) continue;
      codes[x] = __ldg(src + 32 * x);
      words[x] = __ldg(prm + 256 / G * x * p.ldp);
    }
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const int64_t left = rest - 256 * x;
      if (left <= 0) continue;
      const float scale = lo_of(words[x]), zero = hi_of(words[x]);
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // zero + scale * code: the product of 8 and 4 significant bits is exact in FP32.
        const float a = fmaf(scale, static_cast<float>((codes[x] >> (4 * j)) & 15u), zero);
        const float b = fmaf(scale, static_cast<float>((codes[x] >> (4 * j + 16)) & 15u), zero);
        v[j] = pack2(a, b);
      }
      uint16_t* dst = out + 256 * x;
      if (VEC && left >= 8) {
        __stcs(reinterpret_cast<uint4*>(dst), make_uint4(v[0], v[1], v[2], v[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (2 * j < left) dst[2 * j] = static_cast<uint16_t>(v[j]);
          if (2 * j + 1 < left) dst[2 * j + 1] = static_cast<uint16_t>(v[j] >> 16);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ product
// C[m][n] = sum over groups g of  s_gn sum_k x_mk c_nk + z_gn sum_k x_mk,  k in g.
//
// Weights are read once for each 64 rows of X, half a byte each: HBM bounds the call while the
// codes get to the tensor cores without being rounded or passing through shared memory twice.
//   * Columns of W are the 128 rows of a tcgen05.mma and rows of X its narrow operand (16, 32 or 64
//     of them, straight from TMA).  A lane of the expanding warps holds one column's 128 codes of a
//     unit and writes them, as BF16, to tensor memory, from where the MMA reads its A operand.
//   * A code c becomes the BF16 number 16 + c by a shift and one AND-OR for two of them: 16 is the
//     least offset that keeps all four bits of c in a mantissa, and the layout has neighbouring k in
//     the two halves of a word, so that pairs come out in the operand's order.
//   * A group's sums stay apart: D = sum x (16 + c) is read from tensor memory when its group ends, and
//     acc += s D + (z / 16 - s) S, S = sum 16 x, in FP32 (16 s may be past its range where s is not).  S comes
//     from two warps of their own (mma.sync with an operand of 16 throughout); for 64 rows that would take them 2000
//     cycles a unit, and S comes from the same pipe as D, by products with 16 in tensor memory.  Codes and x are
//     exact in BF16, so no weight is rounded.
// Units of 128 columns x 256 k of all column tiles are cut evenly over one CTA per SM; a tile cut between
// CTAs is finished by the last of them to arrive, which adds the parts in CTA order (results do not depend on
// arrival).  More than 64 rows of X: each column tile is computed for one block of 64 after the other,
// by CTAs that run together, so the weights come from L2 after the first.
// Warps: 0-3 groups' sums and joins (a thread per column), 4-11 expansion (a warpgroup for each half of a
// unit), 12 copies, 13 issues products, 14-15 sums of X.
// Measured: 16 rows times 100003 columns of 4096 in 54 us, 4.1 TB/s; without the expansion's arithmetic 49, with
// copies alone 42 (measured on altered copies of this kernel).  A third expanding warpgroup (56 us) and rings of their own for codes, X and
// parameters (59) were slower: more warps share the same logic pipe.
constexpr int kMaxCtas = 160;               // CTAs that the workspace has room for
constexpr int kUnitK = 256, kHalfK = 128;
constexpr uint32_t kCodeBytes = 128 * kUnitK / 2;
constexpr int kEpiWarps = 4;
constexpr uint32_t kMinUnits = 2;           // of a CTA
// Tensor memory: 256 columns of D (and S), buffers of an expanded half of a unit, the operand of S.
constexpr uint32_t kSixteens = 0x41804180u;  // two BF16
constexpr uint32_t kACol = 256, kSumCol = 448, kTmemCols = 512;
constexpr int64_t kCounterBytes = 1024;
static_assert(kMaxCtas * 4 <= kCounterBytes, "counters");

template <int NTOK, int GROUP>
struct Cfg {
  static constexpr bool kSumsByTile = NTOK == 64;            // S by the same pipe as D
  static constexpr int kSumWarps = kSumsByTile ? 0 : 2;
  static constexpr int kProducer = kEpiWarps + 8, kIssuer = kProducer + 1, kFirstSum = kIssuer + 1;
  static constexpr int kThreads = 32 * (kFirstSum + kSumWarps);
  static constexpr int kABuffers = kSumsByTile ? 3 : 4;
  static constexpr int kStages = NTOK == 16 ? 7 : NTOK == 32 ? 6 : 4;
  static constexpr int kGroups = kUnitK / GROUP;             // of a unit
  // Groups whose D is read together: all of a unit where they are at most 128 columns.
  static constexpr int kMost = 128 / NTOK / (kSumsByTile ? 2 : 1), kTogether = kGroups < kMost ? kGroups : kMost;
  static constexpr int kReads = kGroups / kTogether;         // of a unit
  static constexpr int kSlot = kTogether * NTOK * (kSumsByTile ? 2 : 1);  // columns of one
  static constexpr int kSlots = 256 / kSlot < 8 ? 256 / kSlot : 8;
  static_assert(kSlots >= 2 && (kReads == 1 || kReads % 2 == 0), "reads");
  static constexpr uint32_t kXBox = NTOK * 128, kXBytes = 4 * kXBox, kParamBytes = kGroups * 512;
  static constexpr uint32_t kStage = kCodeBytes + kXBytes + 4096;
  static constexpr uint32_t kSumBytes = kSumsByTile ? 0 : kGroups * NTOK * 4;  // of a stage
  static constexpr uint32_t kSmem = 1024 + kStages * (kStage + kSumBytes);
  static_assert(kStage % 1024 == 0 && kParamBytes <= 4096 && kSmem + 1024 <= 227 * 1024, "shared memory, with the static part");
};

struct Control {
  uint64_t full[7], empty[7], sums[7], afull[4], aempty[4], dfull[8], dempty[8], drain;
  uint32_t tmem_base, abort, issued, verdict;
};

// Units cut evenly over workers, the first `rem` of them one unit longer.
struct Split {
  uint32_t q, rem;
  __device__ __forceinline__ Split(uint32_t units, uint32_t workers) : q(units / workers), rem(units - q * workers) {}
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return c * q + (c < rem ? c : rem); }
  __device__ __forceinline__ uint32_t worker(uint32_t x) const {  // that has unit x
    const uint32_t long_units = rem * (q + 1);
    return x < long_units ? x / (q + 1) : rem + (x - long_units) / q;
  }
};

struct Maps {
  CUtensorMap codes, x, params;
};

__device__ __forceinline__ uint32_t take_ticket(uint32_t* a) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a) : "memory");
  return old;
}
__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ uint32_t elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p;
}
// D[tmem] (+)= A[tmem] B[smem]: row m of A in lane m, two BF16 of k per 32-bit column, low half first.  The
// whole warp comes here and its elected lane issues: operands are then uniform over a converged warp, and an
// MMA takes 10 cycles to issue where a branch of one lane took 45 (128 x 16 x 16, one after the other).
template <bool ACCUMULATE>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "n"(ACCUMULATE ? 1 : 0), "r"(lead)
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

__device__ __forceinline__ void tmem_st_x32(uint32_t a, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t a, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

// Codes -> BF16 pairs 16 + code: bits 3-6 of 0x4180.
struct Magic {
  uint32_t mask, offset;  // in registers: as constants the AND and the OR are two instructions
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x00780078;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(offset));
  }
  __device__ __forceinline__ uint32_t pair(uint32_t w) const {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(offset));  // (a & b) | c
    return d;
  }
};

// 16 times the sums of eight rows of X over 16 k: a row of the product with 16 throughout.
__device__ __forceinline__ void mma_sums(float (&c)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%4,%4,%4}, {%5,%6}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(kSixteens), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}

template <int NTOK, int GROUP>
__global__ void __launch_bounds__(Cfg<NTOK, GROUP>::kThreads, 1) gemm_w4_kernel(const __grid_constant__ Maps maps, const W4GemmParams p) {
  using C = Cfg<NTOK, GROUP>;
  constexpr int kABuffers = C::kABuffers, kProducer = C::kProducer, kIssuer = C::kIssuer, kFirstSum = C::kFirstSum;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Control ctl;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u, sum_ring = ring + C::kStages * C::kStage;
  volatile uint32_t* abort = &ctl.abort;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform to the compiler too)

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&ctl.full[s]), 1);
      mbar_init(smem_u32(&ctl.empty[s]), 1 + kEpiWarps);
      if (!C::kSumsByTile) mbar_init(smem_u32(&ctl.sums[s]), C::kSumWarps);
    }
    for (int a = 0; a < kABuffers; ++a) {
      mbar_init(smem_u32(&ctl.afull[a]), 4);
      mbar_init(smem_u32(&ctl.aempty[a]), 1);
    }
    for (int a = 0; a < C::kSlots; ++a) {
      mbar_init(smem_u32(&ctl.dfull[a]), 1);
      mbar_init(smem_u32(&ctl.dempty[a]), kEpiWarps);
    }
    mbar_init(smem_u32(&ctl.drain), 1);
    ctl.abort = 0;
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(&ctl.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProducer && lane < 3) tma_prefetch_map(lane == 0 ? &maps.codes : lane == 1 ? &maps.params : &maps.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, ctl.tmem_base, 0);
  const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);  // this warp's lanes
  if constexpr (C::kSumsByTile) {
    if (warp < kEpiWarps) {
      tmem_st_x8(tl + kSumCol, kSixteens);
      tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }

  const uint32_t kb = static_cast<uint32_t>((p.K + kUnitK - 1) / kUnitK);
  const uint32_t blocks = static_cast<uint32_t>((p.M + NTOK - 1) / NTOK);
  const uint32_t tiles = static_cast<uint32_t>((p.N + 127) / 128) * blocks;
  const Split split(tiles * kb, gridDim.x);
  const uint32_t u0 = split.start(blockIdx.x), n = split.start(blockIdx.x + 1) - u0;

  if (warp == kProducer) {
    // ------------------------------------------------------------ copies: a lane for each of a stage
    uint32_t tile = u0 / kb, k = u0 - tile * kb, col = tile / blocks, row = tile - col * blocks, s = 0, ph = 1, i = 0;
    const int box = lane - 2;  // of X
    const CUtensorMap* map = lane == 0 ? &maps.codes : lane == 1 ? &maps.params : &maps.x;
    const uint32_t to = ring + (lane == 0 ? 0u : lane == 1 ? kCodeBytes + C::kXBytes : kCodeBytes + box * C::kXBox);
    pdl_wait();
    for (; i < n; ++i) {
      if (!mbar_wait_warp(smem_u32(&ctl.empty[s]), ph, abort, p.status, kDevTimeoutProducer)) break;
      const uint32_t f = smem_u32(&ctl.full[s]);
      if (lane == 0) mbar_arrive_expect_tx(f, kCodeBytes + C::kXBytes + C::kParamBytes);
      __syncwarp();
      const int32_t x = lane == 0 ? k * (kUnitK / 2) : lane == 1 ? col * 128 : k * kUnitK + box * 64;
      const int32_t y = lane == 0 ? col * 128 : lane == 1 ? k * C::kGroups : row * NTOK;
      if (lane < 6) tma_load_2d(to + s * C::kStage, map, f, x, y);
      if (++s == C::kStages) s = 0, ph ^= 1u;
      if (++k == kb) {
        k = 0;
        if (++row == blocks) row = 0, ++col;
      }
    }
    pdl_trigger();
    if (lane == 0) ctl.issued = i;
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ products
    constexpr uint32_t idesc = idesc_bf16_f32(128, NTOK, false, false);
    const uint64_t x0 = sdesc_sw128(ring + kCodeBytes, 16, 1024);
    const uint32_t lead = elect();
    uint32_t s = 0, slot = 0, dph = 1, a = 0, aph = 0;
    bool ok = true;
    pdl_wait();  // bounded waits start when this grid's data can arrive
    for (uint32_t i = 0; i < n; ++i) {
      const uint64_t x = x0 + s * (C::kStage >> 4);
#pragma unroll
      for (int r = 0; r < C::kReads; ++r) {
        constexpr int kSteps = GROUP / 16, kHalfReads = C::kReads > 1 ? C::kReads / 2 : 1, kHalves = C::kReads > 1 ? 1 : 2;
        // Lanes wait for different barriers at once, as every wait takes 60 cycles and more: the expanded halves and the place
        // of D.  (The warps that expanded a half have seen its stage filled.)
        const bool half = r % kHalfReads == 0 && lane < kHalves;  // a begins anew with r, and has an even number of buffers then
        const uint32_t bar = half ? smem_u32(&ctl.afull[a + lane]) : smem_u32(&ctl.dempty[slot]);
        ok = mbar_wait_warp(bar, half ? aph : dph, abort, p.status, kDevTimeoutMma);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + slot * C::kSlot;
#pragma unroll
        for (int j = 0; j < C::kTogether * kSteps; ++j) {
          const int step = r * C::kTogether * kSteps + j, in = step % (kHalfK / 16);  // 16 k each: of the unit, of the half
          const uint64_t b = x + ((step >> 2) * C::kXBox + (step & 3) * 32) / 16;
          const uint32_t at = tmem + kACol + 64 * a + (kHalves == 2 ? step / (kHalfK / 16) * 64 : 0) + in * 8;
          if (j % kSteps == 0) umma_ts<false>(d + j / kSteps * NTOK, at, b, idesc, lead);
          else umma_ts<true>(d + j / kSteps * NTOK, at, b, idesc, lead);
        }
        if constexpr (C::kSumsByTile) {
          static_assert(C::kTogether == 1, "S lies behind its D");
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const int step = r * kSteps + j;
            const uint64_t b = x + ((step >> 2) * C::kXBox + (step & 3) * 32) / 16;
            if (j == 0) umma_ts<false>(d + NTOK, tmem + kSumCol, b, idesc, lead);
            else umma_ts<true>(d + NTOK, tmem + kSumCol, b, idesc, lead);
          }
        }
        commit(&ctl.dfull[slot], lead);
        if (++slot == C::kSlots) slot = 0, dph ^= 1u;
        if (r % kHalfReads == kHalfReads - 1) {
#pragma unroll
          for (int e = 0; e < kHalves; ++e) commit(&ctl.aempty[a + e], lead);
          if ((a += kHalves) == kABuffers) a = 0, aph ^= 1u;
        }
      }
      if (!ok) break;
      if (p.fault != 1) commit(&ctl.empty[s], lead);
      if (++s == C::kStages) s = 0;
    }
    commit(&ctl.drain, lead);
    uint32_t never = 0;
    mbar_wait(smem_u32(&ctl.drain), 0, &never, p.status, kDevTimeoutDrain);
    __syncwarp();
  } else if (warp >= kFirstSum) {
    // ------------------------------------------------------------ sums of X: a warp takes every other eight rows
    if constexpr (!C::kSumsByTile) {
    constexpr int kTiles = NTOK / 8 / C::kSumWarps;
    const int w = warp - kFirstSum, r8 = lane & 7, piece = lane >> 3;
    uint32_t s = 0, ph = 0;
    pdl_wait();
    for (uint32_t i = 0; i < n; ++i) {
      if (!mbar_wait_warp(smem_u32(&ctl.full[s]), ph, abort, p.status, kDevTimeoutMma)) break;
      const uint32_t x = ring + s * C::kStage + kCodeBytes + r8 * 128, out = sum_ring + s * C::kSumBytes + lane * 8;
      float c[kTiles][2][4];  // two chains
#pragma unroll
      for (int step = 0; step < kUnitK / 32; ++step) {  // 32 k
        if (step % (GROUP / 32) == 0) {
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) c[t][e][0] = c[t][e][1] = c[t][e][2] = c[t][e][3] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          uint32_t b[4];
          ldmatrix_x4(x + (step >> 1) * C::kXBox + (t * C::kSumWarps + w) * 1024 + ((((step & 1) * 4 + piece) ^ r8) << 4), b);
          mma_sums(c[t][0], b[0], b[1]);
          mma_sums(c[t][1], b[2], b[3]);
        }
        if (step % (GROUP / 32) == GROUP / 32 - 1 && lane < 4) {  // rows of the product are alike
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(out + (step / (GROUP / 32) * NTOK + (t * C::kSumWarps + w) * 8) * 4),
                         "f"(c[t][0][0] + c[t][1][0]), "f"(c[t][0][1] + c[t][1][1])
                         : "memory");
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl.sums[s]));
      if (++s == C::kStages) s = 0, ph ^= 1u;
    }
    }
  } else if (warp >= kEpiWarps) {
    // ------------------------------------------------------------ expansion
    const Magic magic;
    const uint32_t half = (warp - kEpiWarps) / 4, row = (warp & 3) * 32 + lane, swz = row & 7;  // 128-byte rows, 16-byte pieces swizzled
    uint32_t s = 0, ph = 0, a = half, aph = 1;
    pdl_wait();
    for (uint32_t i = 0; i < n; ++i) {
      const uint32_t bar = lane == 0 ? smem_u32(&ctl.full[s]) : smem_u32(&ctl.aempty[a]);
      if (!mbar_wait_warp(bar, lane == 0 ? ph : aph, abort, p.status, kDevTimeoutMma)) break;
      const uint32_t from = ring + s * C::kStage + row * 128, to = tl + kACol + 64 * a;
      uint32_t v[32];
      auto expand = [&](uint32_t c) {  // two pieces
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint4 w = lds128(from + ((half * 4 + c + y) ^ swz) * 16);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[y * 16 + 4 * j] = magic.pair(ws[j] << 3);
            v[y * 16 + 4 * j + 1] = magic.pair(ws[j] >> 1);
            v[y * 16 + 4 * j + 2] = magic.pair(ws[j] >> 5);
            v[y * 16 + 4 * j + 3] = magic.pair(ws[j] >> 9);
          }
        }
      };
      expand(0);
      tc_fence_after();
      tmem_st_x32(to, v);
      expand(2);
      tmem_st_x32(to + 32, v);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl.afull[a]));
      if (++s == C::kStages) s = 0, ph ^= 1u;
      if ((a += 2) >= kABuffers) a -= kABuffers, aph ^= 1u;
    }
  } else {
    // ------------------------------------------------------------ groups' sums, and the tiles' join
    const int col = warp * 32 + lane;
    uint32_t* counters = static_cast<uint32_t*>(p.ws);
    float4* parts = reinterpret_cast<float4*>(static_cast<uint8_t*>(p.ws) + kCounterBytes);
    uint32_t i = 0, s = 0, ph = 0, slot = 0, dph = 0;
    pdl_wait();
    while (i < n) {
      const uint32_t tile = (u0 + i) / kb, first = tile * kb, k0 = u0 + i - first, units = min(kb - k0, n - i);
      float acc[NTOK];
#pragma unroll
      for (int t = 0; t < NTOK; ++t) acc[t] = 0.f;
      bool ok = true;
      for (const uint32_t to = i + units; ok && i < to; ++i) {
#pragma unroll
        for (int r = 0; r < C::kReads; ++r) {
          // The stage (its parameters), the sums of X, D.
          const bool first = r == 0 && lane < (C::kSumsByTile ? 1 : 2);
          const uint32_t bar = first ? (lane == 0 ? smem_u32(&ctl.full[s]) : smem_u32(&ctl.sums[s])) : smem_u32(&ctl.dfull[slot]);
          ok = mbar_wait_warp(bar, first ? ph : dph, abort, p.status, kDevTimeoutEpilogue);
          if (!ok) break;
          tc_fence_after();
          constexpr int kCols = C::kTogether * NTOK, kAtOnce = kCols < 32 || C::kSumsByTile ? 16 : 32;
          const uint32_t d = tl + slot * C::kSlot;
#pragma unroll
          for (int c = 0; c < kCols; c += kAtOnce) {
            uint32_t dv[kAtOnce], sv[C::kSumsByTile ? kAtOnce : 1];
            if constexpr (kAtOnce == 16) tmem_ld_32x32b_x16(d + c, dv);
            else tmem_ld_32x32b_x32(d + c, dv);
            if constexpr (C::kSumsByTile) tmem_ld_32x32b_x16(d + NTOK + c, sv);
            tmem_ld_wait();
            if (c + kAtOnce == kCols) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&ctl.dempty[slot]));
            }
#pragma unroll
            for (int t = 0; t < kAtOnce; t += 4) {
              const int g = r * C::kTogether + (c + t) / NTOK, tok = (c + t) % NTOK;
              const uint32_t prm = lds32(ring + s * C::kStage + kCodeBytes + C::kXBytes + g * 512 + col * 4);
              const float scale = lo_of(prm), zero = hi_of(prm) * 0.0625f - scale;
              uint4 x;
              if constexpr (C::kSumsByTile) x = make_uint4(sv[t], sv[t + 1], sv[t + 2], sv[t + 3]);
              else x = lds128(sum_ring + s * C::kSumBytes + (g * NTOK + tok) * 4);
              acc[tok] = fmaf(scale, __uint_as_float(dv[t]), fmaf(zero, __uint_as_float(x.x), acc[tok]));
              acc[tok + 1] = fmaf(scale, __uint_as_float(dv[t + 1]), fmaf(zero, __uint_as_float(x.y), acc[tok + 1]));
              acc[tok + 2] = fmaf(scale, __uint_as_float(dv[t + 2]), fmaf(zero, __uint_as_float(x.z), acc[tok + 2]));
              acc[tok + 3] = fmaf(scale, __uint_as_float(dv[t + 3]), fmaf(zero, __uint_as_float(x.w), acc[tok + 3]));
            }
          }
          if (++slot == C::kSlots) slot = 0, dph ^= 1u;
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(smem_u32(&ctl.empty[s]));
        if (++s == C::kStages) s = 0, ph ^= 1u;
      }
      // One decision of the four warps, so that none is left alone in a barrier.
      if (!ok) *abort = 1;
      epi_bar();
      if (threadIdx.x == 0) ctl.verdict = *abort;
      epi_bar();
      if (ctl.verdict) break;
      const int64_t m0 = static_cast<int64_t>(tile % blocks) * NTOK, c0 = static_cast<int64_t>(tile / blocks) * 128 + col;
      const int m = static_cast<int>(p.M - m0 < NTOK ? p.M - m0 : NTOK), nq = (m + 3) / 4;
      bool write = units == kb;
      if (!write) {
        // A part of a tile of several CTAs: [4 rows of X][column] float4.  A CTA has at most two, the one
        // that its share begins in and the one that it ends in, and is the first of at most one.
        auto part_of = [&](uint32_t c) {
          return parts + (static_cast<int64_t>(c) * 2 + (split.start(c) >= first ? 0 : 1)) * (NTOK / 4) * 128 + col;
        };
        float4* mine = part_of(blockIdx.x);
#pragma unroll
        for (int q = 0; q < NTOK / 4; ++q)
          if (q < nq) __stcg(mine + q * 128, make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]));
        const uint32_t lo = split.worker(first), hi = split.worker(first + kb - 1);
        epi_bar();  // the ticket's release covers the four warps' stores
        if (threadIdx.x == 0) {
          const bool last = take_ticket(counters + lo) == hi - lo;
          if (last) counters[lo] = 0;  // all tickets are taken: ready for the next call
          ctl.verdict = last;
        }
        epi_bar();
        write = ctl.verdict != 0;
        if (write) {
#pragma unroll
          for (int t = 0; t < NTOK; ++t) acc[t] = 0.f;
          constexpr int kChunk = NTOK / 4 < 8 ? NTOK / 4 : 8;  // loads in flight: registers
#pragma unroll
          for (int q0 = 0; q0 < NTOK / 4; q0 += kChunk) {
            if (q0 >= nq) break;
#pragma unroll NTOK == 16 ? 2 : 1
            for (uint32_t c = lo; c <= hi; ++c) {
              const float4* src = part_of(c);
              float4 v[kChunk];
#pragma unroll
              for (int q = 0; q < kChunk; ++q) v[q] = q0 + q < nq ? __ldcg(src + (q0 + q) * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int q = 0; q < kChunk; ++q) {
                float* to = &acc[4 * (q0 + q)];
                to[0] += v[q].x;
                to[1] += v[q].y;
                to[2] += v[q].z;
                to[3] += v[q].w;
              }
            }
          }
        }
      }
      if (write && c0 < p.N) {
        if (p.c_f32) {
          float* to = static_cast<float*>(p.C) + m0 * p.ldc + c0;
#pragma unroll
          for (int t = 0; t < NTOK; ++t)
            if (t < m) to[t * p.ldc] = acc[t];
        } else {
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.C) + m0 * p.ldc + c0;
#pragma unroll
          for (int t = 0; t < NTOK; ++t)
            if (t < m) to[t * p.ldc] = __float2bfloat16_rn(acc[t]);
        }
      }
      epi_bar();  // verdict is written again only after all have read it
    }
  }

  tc_fence_before();
  __syncthreads();
  if (ctl.abort && warp == kProducer && lane == 0) {
    // Some wait ran out: the copies in flight land before the CTA ends.
    const uint32_t issued = ctl.issued;
    uint32_t never = 0;
    for (uint32_t j = issued > C::kStages ? issued - C::kStages : 0u; j < issued; ++j)
      mbar_wait(smem_u32(&ctl.full[j % C::kStages]), (j / C::kStages) & 1u, &never, p.status, kDevTimeoutDrain);
  }
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int NTOK, int GROUP>
cudaError_t launch_variant(const W4GemmParams& p, int sms, cudaStream_t s) {
  using C = Cfg<NTOK, GROUP>;
  Maps m;
  // A single row has no stride of its own.
  const int64_t words = (p.K + 7) / 8, ldq = p.N > 1 ? p.ldq : (4 * words + 15) / 16 * 16, ldx = p.M > 1 ? p.ldx : (p.K + 7) / 8 * 8;
  const int64_t groups = (p.K + GROUP - 1) / GROUP, ldp = groups > 1 ? p.ldp : (p.N + 3) / 4 * 4;
  if (!make_tile_map(&m.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.Q, 4 * words, p.N, ldq, 1, 0, kUnitK / 2, 128,
                     CU_TENSOR_MAP_SWIZZLE_128B, 1) ||
      !make_tile_map(&m.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.X, p.K, p.M, ldx, 1, 0, 64, NTOK, CU_TENSOR_MAP_SWIZZLE_128B, 1) ||
      !make_tile_map(&m.params, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, p.params, p.N, groups, ldp, 1, 0, 128, C::kGroups,
                     CU_TENSOR_MAP_SWIZZLE_NONE, 1))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> attr_done{0};
  const cudaError_t e = ensure_smem_attr(gemm_w4_kernel<NTOK, GROUP>, C::kSmem, attr_done);
  if (e != cudaSuccess) return e;
  const int64_t units = (p.N + 127) / 128 * ((p.M + NTOK - 1) / NTOK) * ((p.K + kUnitK - 1) / kUnitK);
  int64_t ctas = (units + kMinUnits - 1) / kMinUnits;
  if (ctas > sms) ctas = sms;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  W4GemmParams q = p;
  q.fault = g_fault_injection;
  return launch_pdl(gemm_w4_kernel<NTOK, GROUP>, dim3(static_cast<unsigned>(ctas)), dim3(C::kThreads), C::kSmem, s, m, q);
}

template <int NTOK>
cudaError_t launch_ntok(const W4GemmParams& p, int sms, cudaStream_t s) {
  return p.group == 32   ? launch_variant<NTOK, 32>(p, sms, s)
         : p.group == 64 ? launch_variant<NTOK, 64>(p, sms, s)
                         : launch_variant<NTOK, 128>(p, sms, s);
}

int ntok_of(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

}  // namespace

#define DG_W4_ROWS(KERNEL, G, VEC)                                                              \
  if (group == G && vec == VEC)                                                                \
    return big ? launch_pdl(KERNEL<G, VEC, 4>, g, b, 0, s, p, pieces) : launch_pdl(KERNEL<G, VEC, 1>, g, b, 0, s, p, pieces);
#define DG_W4_ALL(KERNEL)                                                                      \
  auto count = [&](int words) { return p.N * (((p.K + 7) / 8 + words - 1) / words); };         \
  const bool big = count(128) >= static_cast<int64_t>(sms) * 128;                              \
  const int64_t pieces = count(big ? 128 : 32), need = (pieces + kThreads / 32 - 1) / (kThreads / 32), cap = static_cast<int64_t>(sms) * 64; \
  const dim3 g(static_cast<unsigned>(need < cap ? need : cap)), b(kThreads);                   \
  DG_W4_ROWS(KERNEL, 32, true)                                                                 \
  DG_W4_ROWS(KERNEL, 32, false)                                                                \
  DG_W4_ROWS(KERNEL, 64, true)                                                                 \
  DG_W4_ROWS(KERNEL, 64, false)                                                                \
  DG_W4_ROWS(KERNEL, 128, true)                                                                \
  DG_W4_ROWS(KERNEL, 128, false)                                                               \
  return cudaErrorInvalidValue;

cudaError_t launch_quantize_w4(const W4RowsParams& p, int group, bool vec, int sms, cudaStream_t s) { DG_W4_ALL(quantize_w4_kernel) }

cudaError_t launch_dequantize_w4(const W4RowsParams& p, int group, bool vec, int sms, cudaStream_t s) { DG_W4_ALL(dequantize_w4_kernel) }
#undef DG_W4_ROWS
#undef DG_W4_ALL

int64_t gemm_w4_ws_bytes(int64_t M, int64_t N, int64_t K) {
  // Units are counted in 31 bits.
  const int64_t rows = (M + 63) / 64, tiles = (N + 127) / 128, kb = (K + kUnitK - 1) / kUnitK;
  if (rows > INT32_MAX / tiles / kb) return 0;
  return kCounterBytes + int64_t(kMaxCtas) * 2 * ntok_of(M) * 128 * 4;
}

cudaError_t launch_gemm_w4(const W4GemmParams& p, int sms, cudaStream_t s) {
  const int ntok = ntok_of(p.M);
  return ntok == 16 ? launch_ntok<16>(p, sms, s) : ntok == 32 ? launch_ntok<32>(p, sms, s) : launch_ntok<64>(p, sms, s);
}

}  // namespace dg
