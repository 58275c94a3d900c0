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
// A lane holds 8 elements, one word of codes; G / 8 neighbouring lanes hold a group, so that a warp
// reads 512 contiguous bytes and writes 128.
template <int G, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_w4_kernel(const W4RowsParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t words = (p.K + 7) / 8, per_row = (words + 31) / 32;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < p.N * per_row; i += warps) {
    const int64_t n = i / per_row, w = (i - n * per_row) * 32 + lane;
    const uint16_t* src = p.W + n * p.ldw + 8 * w;
    const int64_t left = p.K - 8 * w;  // elements of this word: 8, fewer at the row's end, none past it
    uint32_t v[4];
    if (VEC && left >= 8) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(src));
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = 2 * j < left ? src[2 * j] : 0, b = 2 * j + 1 < left ? src[2 * j + 1] : 0;
        v[j] = a | b << 16;
      }
    }
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (2 * j < left) lo = fminf(lo, lo_of(v[j])), hi = fmaxf(hi, lo_of(v[j]));
      if (2 * j + 1 < left) lo = fminf(lo, hi_of(v[j])), hi = fmaxf(hi, hi_of(v[j]));
    }
#pragma unroll
    for (int o = G / 16; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
    }
    if (left <= 0) continue;
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float scale = __bfloat162float(sb);
    uint32_t codes = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = k & 1 ? hi_of(v[k >> 1]) : lo_of(v[k >> 1]);
      const float q = scale > 0.f && k < left ? rintf(__fdiv_rn(__fsub_rn(x, lo), scale)) : 0.f;
      codes |= static_cast<uint32_t>(fminf(fmaxf(q, 0.f), 15.f)) << code_at(k);
    }
    reinterpret_cast<uint32_t*>(p.Q + n * p.ldq)[w] = codes;
    if (lane % (G / 8) == 0)
      p.params[8 * w / G * p.ldp + n] =
          static_cast<uint32_t>(__bfloat16_as_ushort(sb)) | (__float_as_uint(lo) & 0xFFFF0000u);
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads) dequantize_w4_kernel(const W4RowsParams p, const int group_words) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t words = (p.K + 7) / 8, per_row = (words + 31) / 32;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < p.N * per_row; i += warps) {
    const int64_t n = i / per_row, w = (i - n * per_row) * 32 + lane;
    if (w >= words) continue;
    const uint32_t codes = reinterpret_cast<const uint32_t*>(p.Q + n * p.ldq)[w];
    const uint32_t prm = p.params[w / group_words * p.ldp + n];
    const float scale = lo_of(prm), zero = hi_of(prm);
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // zero + scale * code: the product of 8 and 4 significant bits is exact in FP32.
      const float a = fmaf(scale, static_cast<float>((codes >> (4 * j)) & 15u), zero);
      const float b = fmaf(scale, static_cast<float>((codes >> (4 * j + 16)) & 15u), zero);
      v[j] = pack2(a, b);
    }
    uint16_t* dst = p.W + n * p.ldw + 8 * w;
    const int64_t left = p.K - 8 * w;
    if (VEC && left >= 8) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (2 * j < left) dst[2 * j] = static_cast<uint16_t>(v[j]);
        if (2 * j + 1 < left) dst[2 * j + 1] = static_cast<uint16_t>(v[j] >> 16);
      }
    }
  }
}

dim3 rows_grid(const W4RowsParams& p, int sms) {
  const int64_t need = (p.N * (((p.K + 7) / 8 + 31) / 32) + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(sms) * 8;
  return dim3(static_cast<unsigned>(need < cap ? need : cap));
}

// ------------------------------------------------------------------ product
// One warp per output column, its lanes over the words of the column, eight rows of X at a time.
__global__ void __launch_bounds__(kThreads) gemm_w4_kernel(const W4GemmParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t words = (p.K + 7) / 8;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t n = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); n < p.N; n += warps) {
    for (int64_t m0 = 0; m0 < p.M; m0 += 8) {
      float acc[8] = {};
      for (int64_t w = lane; w < words; w += 32) {
        const uint32_t codes = reinterpret_cast<const uint32_t*>(p.Q + n * p.ldq)[w];
        const uint32_t prm = p.params[8 * w / p.group * p.ldp + n];
        const float scale = lo_of(prm), zero = hi_of(prm);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (8 * w + k >= p.K) break;
          const float v = fmaf(scale, static_cast<float>((codes >> code_at(k)) & 15u), zero);
#pragma unroll
          for (int m = 0; m < 8; ++m)
            if (m0 + m < p.M) acc[m] = fmaf(v, __uint_as_float(static_cast<uint32_t>(p.X[(m0 + m) * p.ldx + 8 * w + k]) << 16), acc[m]);
        }
      }
#pragma unroll
      for (int m = 0; m < 8; ++m) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(~0u, acc[m], o);
        if (lane != 0 || m0 + m >= p.M) continue;
        if (p.c_f32) static_cast<float*>(p.C)[(m0 + m) * p.ldc + n] = acc[m];
        else static_cast<__nv_bfloat16*>(p.C)[(m0 + m) * p.ldc + n] = __float2bfloat16_rn(acc[m]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_quantize_w4(const W4RowsParams& p, int group, bool vec, int sms, cudaStream_t s) {
  const dim3 g = rows_grid(p, sms), b(kThreads);
#define DG_W4_CASE(G) \
  if (group == G) return vec ? launch_pdl(quantize_w4_kernel<G, true>, g, b, 0, s, p) : launch_pdl(quantize_w4_kernel<G, false>, g, b, 0, s, p);
  DG_W4_CASE(32)
  DG_W4_CASE(64)
  DG_W4_CASE(128)
#undef DG_W4_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_dequantize_w4(const W4RowsParams& p, int group, bool vec, int sms, cudaStream_t s) {
  const dim3 g = rows_grid(p, sms), b(kThreads);
  return vec ? launch_pdl(dequantize_w4_kernel<true>, g, b, 0, s, p, group / 8)
             : launch_pdl(dequantize_w4_kernel<false>, g, b, 0, s, p, group / 8);
}

int64_t gemm_w4_ws_bytes(int64_t, int64_t, int64_t) { return 256; }

cudaError_t launch_gemm_w4(const W4GemmParams& p, int sms, cudaStream_t s) {
  const int64_t need = (p.N + kThreads / 32 - 1) / (kThreads / 32), cap = static_cast<int64_t>(sms) * 8;
  return launch_pdl(gemm_w4_kernel, dim3(static_cast<unsigned>(need < cap ? need : cap)), dim3(kThreads), 0, s, p);
}

}  // namespace dg
