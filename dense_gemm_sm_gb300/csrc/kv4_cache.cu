// kv4_cache.cu -- writing rows of keys and values into the paged 4-bit cache, and reading them
// back as BF16.  Per row x of d elements (one token, one head):
//   zero = min x,  scale = bf16((max x - min x) / 15),
//   code_c = clamp(rne((x_c - zero) / scale), 0, 15),  x_c ~ zero + scale * code_c.
// The minimum of BF16 values is one of them, so zero is exact in BF16; the scale is rounded
// before the codes are taken, so a code is the nearest one of the values that will be read.
// Differences, divisions and roundings are IEEE FP32 operations; a constant row has scale 0
// and codes 0.
//
// HBM-bound: 4 d bytes of K and V on one side, d + 8 on the other, per (token, head).  A warp
// takes one token and a run of its heads, several at a time with their loads together: lanes 0-15
// the key's row, lanes 16-31 the value's, d / 16 elements a lane (16-byte accesses at d = 128).
// Writing is bound by its instructions, so they are few: what a token needs once (its slot's
// page) is found once; minimum and maximum are reduced together as one BF16 pair (maximum,
// -minimum); quotients come from a reciprocal, correctly rounded by one step with their exact
// remainder; codes are put together by FP32 multiply-adds.  8192 tokens of 8 heads written and
// read back: 51 us with a warp per (token, head), 64-bit indices and the compiler's divisions
// (450 instructions for each), 32 us with a reciprocal whose halves were set right afterwards.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

// Small CTAs, so that what does not fill the last wave is little: 8192 tokens of 8 heads written and
// read back take 23.3 us, with 256 threads 26.1 (64: 23.1, but 2000 tokens 12.4 and not 10.6).
constexpr int kThreads = 128;

// Byte offset, in its record, of the two-byte piece of V codes that holds columns
// [4 m, 4 m + 4) of token u (0..15).
template <int D>
__device__ __forceinline__ int v_piece(int u, int m) {
  constexpr int kPer = D / 32;  // pieces of one column group of D / 8
  const int g = m / kPer, j = m - g * kPer;
  return (((u >> 3) * 8 + g) * 4 + ((u & 7) >> 1)) * (D / 8) + j * 4 + (u & 1) * 2;
}

// The record of a slot, for head 0, and its token's place there; heads are `stride` bytes apart.
template <int D>
__device__ __forceinline__ uint8_t* record_of(const Kv4Params& p, int64_t slot, int* u) {
  const uint64_t n = static_cast<uint64_t>(slot);
  const uint64_t page = n >> 32 ? n / static_cast<uint32_t>(p.page_size)
                                : static_cast<uint32_t>(n) / static_cast<uint32_t>(p.page_size);
  const int in = static_cast<int>(n - page * p.page_size);
  *u = in & 15;
  return p.data + (page * p.heads * (p.page_size / kKv4Tokens) + (in >> 4)) * kv4_record_bytes(D);
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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

// H: heads of a token in flight; a warp's run of heads is a multiple of it.
template <int D, bool VEC, int H>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4Params p, const int heads_per_warp) {
  constexpr int N = D / 16;  // elements of a lane
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const int h0 = blockIdx.y * heads_per_warp, h1 = min(p.heads, h0 + heads_per_warp);
  const int64_t stride = static_cast<int64_t>(p.page_size / kKv4Tokens) * kv4_record_bytes(D);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t token = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); token < p.tokens;
       token += warps) {
    const int64_t slot = p.slots[token];
    if (slot < 0) continue;
    if (slot >= p.pages * p.page_size) {
      if (lane == 0) atomicCAS(p.index_word, 0u, kDevBadIndex);
      continue;
    }
    const uint16_t* row = (is_v ? p.V + token * p.ldv : p.K + token * p.ldk) + l * N;
    int u;
    uint8_t* rec0 = record_of<D>(p, slot, &u);
    int piece[N / 4];
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
      piece[j] = is_v ? 8 * D + v_piece<D>(u, l * (N / 4) + j) : u * (D / 2) + (l * (N / 4) + j) * 2;
    for (int h = h0; h < h1; h += H) {
      uint32_t w[H][N / 2];
#pragma unroll
      for (int x = 0; x < H; ++x) {
        const uint16_t* src = row + (h + x) * D;
        if (VEC) {
          if (N == 8) {
            const uint4 q = *reinterpret_cast<const uint4*>(src);
            w[x][0] = q.x; w[x][1] = q.y; w[x][N / 2 - 2] = q.z; w[x][N / 2 - 1] = q.w;
          } else {
            const uint2 q = *reinterpret_cast<const uint2*>(src);
            w[x][0] = q.x; w[x][1] = q.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < N / 2; ++j) w[x][j] = src[2 * j] | (static_cast<uint32_t>(src[2 * j + 1]) << 16);
        }
      }
#pragma unroll
      for (int x = 0; x < H; ++x) {
        uint32_t hi2 = w[x][0], lo2 = w[x][0];
#pragma unroll
        for (int j = 1; j < N / 2; ++j) {
          hi2 = max2(hi2, w[x][j]);
          lo2 = min2(lo2, w[x][j]);
        }
        // (maximum, -minimum) of the lane's elements, then of the row.
        uint32_t ext = max2(__byte_perm(hi2, lo2, 0x5410) ^ 0x80000000u, __byte_perm(hi2, lo2, 0x7632) ^ 0x80000000u);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ext = max2(ext, __shfl_xor_sync(0xffffffffu, ext, o));
        const float hi = __uint_as_float(ext << 16), lo = __uint_as_float((ext & 0xFFFF0000u) ^ 0x80000000u);
        const float range = __fsub_rn(hi, lo);
        const bool plain = range >= 1e-30f;  // nothing below underflows
        const __nv_bfloat16 sb =
            __float2bfloat16_rn(plain ? quotient(range, 15.f, 1.f / 15.f) : __fdiv_rn(range, 15.f));
        const float scale = __bfloat162float(sb);
        uint32_t codes;
        if (plain) {
          // A quotient is at most 15 (1 + 2^-8): rounded, at most 15.
          const float inv = __frcp_rn(scale);
          constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
          float n[N];
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float v = __uint_as_float(j & 1 ? w[x][j / 2] & 0xFFFF0000u : w[x][j / 2] << 16);
            n[j] = (quotient(__fsub_rn(v, lo), scale, inv) + kRound) - kRound;
          }
#pragma unroll
          for (int j = 0; j < N; j += 4) n[j] = fmaf(fmaf(n[j + 3], 16.f, n[j + 2]), 256.f, fmaf(n[j + 1], 16.f, n[j]));
          // Four codes make an integer below 2^16: the low half of 2^23 + it.
          codes = __float_as_uint(n[0] + 8388608.f) & 0xFFFFu;
          if (N == 8) codes = __byte_perm(codes, __float_as_uint(n[N - 4] + 8388608.f), 0x5410);
        } else {
          codes = 0;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float v = __uint_as_float(j & 1 ? w[x][j / 2] & 0xFFFF0000u : w[x][j / 2] << 16);
            const float q = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(v, lo), scale)) : 0.f;
            codes |= static_cast<uint32_t>(fminf(fmaxf(q, 0.f), 15.f)) << (4 * j);
          }
        }
        // Pieces of two bytes (four columns): a K row's lie together, V's in its own order.
        uint8_t* rec = rec0 + (h + x) * stride;
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
          *reinterpret_cast<uint16_t*>(rec + piece[j]) = static_cast<uint16_t>(codes >> (16 * j));
        if (l == 0)
          *reinterpret_cast<uint32_t*>(rec + 16 * D + (is_v ? 64 : 0) + u * 4) =
              static_cast<uint32_t>(__bfloat16_as_ushort(sb)) | (__float_as_uint(lo) & 0xFFFF0000u);
      }
    }
  }
}

template <int D, bool VEC, int H>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const Kv4Params p, const int heads_per_warp) {
  constexpr int N = D / 16;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const int h0 = blockIdx.y * heads_per_warp, h1 = min(p.heads, h0 + heads_per_warp);
  const int64_t stride = static_cast<int64_t>(p.page_size / kKv4Tokens) * kv4_record_bytes(D);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t token = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); token < p.tokens;
       token += warps) {
    const int64_t slot = p.slots[token];
    const bool past = slot >= p.pages * p.page_size, have = slot >= 0 && !past;
    if (past && lane == 0) atomicCAS(p.index_word, 0u, kDevBadIndex);
    int u = 0;
    const uint8_t* rec0 = have ? record_of<D>(p, slot, &u) : p.data;
    uint16_t* row = (is_v ? p.V + token * p.ldv : p.K + token * p.ldk) + l * N;
    int piece[N / 4];
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
      piece[j] = is_v ? 8 * D + v_piece<D>(u, l * (N / 4) + j) : u * (D / 2) + (l * (N / 4) + j) * 2;
    for (int h = h0; h < h1; h += H) {
      uint32_t codes[H], prm[H];
#pragma unroll
      for (int x = 0; x < H; ++x) {
        codes[x] = prm[x] = 0;  // the value 0
        if (!have) continue;
        const uint8_t* rec = rec0 + (h + x) * stride;
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
          codes[x] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(rec + piece[j])) << (16 * j);
        prm[x] = *reinterpret_cast<const uint32_t*>(rec + 16 * D + (is_v ? 64 : 0) + u * 4);
      }
#pragma unroll
      for (int x = 0; x < H; ++x) {
        const float scale = __uint_as_float(prm[x] << 16), zero = __uint_as_float(prm[x] & 0xFFFF0000u);
        uint32_t w[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          // zero + scale * code: the product of 8 and 4 significant bits is exact in FP32.
          const float a = fmaf(scale, static_cast<float>((codes[x] >> (8 * j)) & 15u), zero);
          const float b = fmaf(scale, static_cast<float>((codes[x] >> (8 * j + 4)) & 15u), zero);
          const __nv_bfloat162 ab = __floats2bfloat162_rn(a, b);
          w[j] = *reinterpret_cast<const uint32_t*>(&ab);
        }
        uint16_t* y = row + (h + x) * D;
        if (VEC) {
          if (N == 8) *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[N / 2 - 2], w[N / 2 - 1]);
          else *reinterpret_cast<uint2*>(y) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
          for (int j = 0; j < N / 2; ++j) {
            y[2 * j] = static_cast<uint16_t>(w[j]);
            y[2 * j + 1] = static_cast<uint16_t>(w[j] >> 16);
          }
        }
      }
    }
  }
}

// Heads of a warp: all of them where the tokens alone fill the GPU's warps, one where they are few.
struct Shape {
  dim3 grid;
  int heads_per_warp, in_flight;
};
Shape shape_of(const Kv4Params& p, int sms, int most) {
  const int64_t slots = static_cast<int64_t>(sms) * 64;  // resident warps
  int64_t runs = slots / (p.tokens < slots ? p.tokens : slots);
  if (runs > p.heads) runs = p.heads;
  Shape s;
  s.heads_per_warp = static_cast<int>((p.heads + runs - 1) / runs);
  s.in_flight = p.heads % most == 0 && s.heads_per_warp >= most ? most : p.heads % 4 == 0 && s.heads_per_warp >= 4 ? 4 : 1;
  s.heads_per_warp = (s.heads_per_warp + s.in_flight - 1) / s.in_flight * s.in_flight;
  const int64_t need = (p.tokens + kThreads / 32 - 1) / (kThreads / 32), cap = static_cast<int64_t>(sms) * 16;
  s.grid = dim3(static_cast<unsigned>(need < cap ? need : cap),
                static_cast<unsigned>((p.heads + s.heads_per_warp - 1) / s.heads_per_warp));
  return s;
}

}  // namespace

#define DG_KV4_LAUNCH(KERNEL, D, VEC, MOST)                                                           \
  (f.in_flight == MOST ? launch_pdl(KERNEL<D, VEC, MOST>, f.grid, b, 0, s, p, f.heads_per_warp)     \
   : f.in_flight == 4  ? launch_pdl(KERNEL<D, VEC, 4>, f.grid, b, 0, s, p, f.heads_per_warp)        \
                       : launch_pdl(KERNEL<D, VEC, 1>, f.grid, b, 0, s, p, f.heads_per_warp))

cudaError_t launch_kv4_append(const Kv4Params& p, int d, bool vec, int sms, cudaStream_t s) {
  const Shape f = shape_of(p, sms, 4);
  const dim3 b(kThreads);
  if (d == 128)
    return vec ? DG_KV4_LAUNCH(kv4_append_kernel, 128, true, 4) : DG_KV4_LAUNCH(kv4_append_kernel, 128, false, 4);
  return vec ? DG_KV4_LAUNCH(kv4_append_kernel, 64, true, 4) : DG_KV4_LAUNCH(kv4_append_kernel, 64, false, 4);
}

cudaError_t launch_kv4_gather(const Kv4Params& p, int d, bool vec, int sms, cudaStream_t s) {
  const Shape f = shape_of(p, sms, 8);
  const dim3 b(kThreads);
  if (d == 128)
    return vec ? DG_KV4_LAUNCH(kv4_gather_kernel, 128, true, 8) : DG_KV4_LAUNCH(kv4_gather_kernel, 128, false, 8);
  return vec ? DG_KV4_LAUNCH(kv4_gather_kernel, 64, true, 8) : DG_KV4_LAUNCH(kv4_gather_kernel, 64, false, 8);
}
#undef DG_KV4_LAUNCH

}  // namespace dg
