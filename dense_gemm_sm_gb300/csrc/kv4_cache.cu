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
// takes one (token, head): lanes 0-15 the key's row, lanes 16-31 the value's, d / 16 elements
// a lane (16-byte accesses at d = 128).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

constexpr int kThreads = 256;

// Byte offset, in its record, of the two-byte piece of V codes that holds columns
// [4 m, 4 m + 4) of token u (0..15).
template <int D>
__device__ __forceinline__ int v_piece(int u, int m) {
  constexpr int kPer = D / 32;  // pieces of one column group of D / 8
  const int g = m / kPer, j = m - g * kPer;
  return (((u >> 3) * 8 + g) * 4 + ((u & 7) >> 1)) * (D / 8) + j * 4 + (u & 1) * 2;
}

template <int D>
__device__ __forceinline__ uint8_t* record_of(const Kv4Params& p, int64_t slot, int head, int* u) {
  const int64_t page = slot / p.page_size;
  const int in = static_cast<int>(slot - page * p.page_size);
  *u = in & 15;
  return p.data + ((page * p.heads + head) * (p.page_size / kKv4Tokens) + (in >> 4)) * kv4_record_bytes(D);
}

template <int D, bool VEC>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4Params p) {
  constexpr int N = D / 16;  // elements of a lane
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const int64_t rows = p.tokens * p.heads;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < rows; i += warps) {
    const int64_t token = i / p.heads;
    const int head = static_cast<int>(i - token * p.heads);
    const int64_t slot = p.slots[token];
    if (slot < 0) continue;
    if (slot >= p.pages * p.page_size) {
      if (lane == 0) atomicCAS(p.index_word, 0u, kDevBadIndex);
      continue;
    }
    const uint16_t* x = (is_v ? p.V + token * p.ldv : p.K + token * p.ldk) + head * D + l * N;
    float v[N];
    if (VEC) {
      uint32_t w[N / 2];
      if (N == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(x);
        w[0] = q.x; w[1] = q.y; w[N / 2 - 2] = q.z; w[N / 2 - 1] = q.w;
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(x);
        w[0] = q.x; w[1] = q.y;
      }
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = __uint_as_float(static_cast<uint32_t>(x[j]) << 16);
    }
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int j = 1; j < N; ++j) {
      lo = fminf(lo, v[j]);
      hi = fmaxf(hi, v[j]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float scale = __bfloat162float(sb);
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float q = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(v[j], lo), scale)) : 0.f;
      codes |= static_cast<uint32_t>(fminf(fmaxf(q, 0.f), 15.f)) << (4 * j);
    }
    int u;
    uint8_t* rec = record_of<D>(p, slot, head, &u);
    if (!is_v) {
      if (N == 8) *reinterpret_cast<uint32_t*>(rec + u * (D / 2) + l * 4) = codes;
      else *reinterpret_cast<uint16_t*>(rec + u * (D / 2) + l * 2) = static_cast<uint16_t>(codes);
    } else {
#pragma unroll
      for (int j = 0; j < N / 4; ++j)
        *reinterpret_cast<uint16_t*>(rec + 8 * D + v_piece<D>(u, l * (N / 4) + j)) =
            static_cast<uint16_t>(codes >> (16 * j));
    }
    if (l == 0)
      *reinterpret_cast<uint32_t*>(rec + 16 * D + (is_v ? 64 : 0) + u * 4) =
          static_cast<uint32_t>(__bfloat16_as_ushort(sb)) | (__float_as_uint(lo) & 0xFFFF0000u);
  }
}

template <int D, bool VEC>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const Kv4Params p) {
  constexpr int N = D / 16;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const int64_t rows = p.tokens * p.heads;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < rows; i += warps) {
    const int64_t token = i / p.heads;
    const int head = static_cast<int>(i - token * p.heads);
    const int64_t slot = p.slots[token];
    uint32_t codes = 0;
    float scale = 0.f, zero = 0.f;
    if (slot >= p.pages * p.page_size) {
      if (lane == 0) atomicCAS(p.index_word, 0u, kDevBadIndex);
    } else if (slot >= 0) {
      int u;
      const uint8_t* rec = record_of<D>(p, slot, head, &u);
      if (!is_v) {
        if (N == 8) codes = *reinterpret_cast<const uint32_t*>(rec + u * (D / 2) + l * 4);
        else codes = *reinterpret_cast<const uint16_t*>(rec + u * (D / 2) + l * 2);
      } else {
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
          codes |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(rec + 8 * D + v_piece<D>(u, l * (N / 4) + j)))
                   << (16 * j);
      }
      const uint32_t prm = *reinterpret_cast<const uint32_t*>(rec + 16 * D + (is_v ? 64 : 0) + u * 4);
      scale = __uint_as_float(prm << 16);
      zero = __uint_as_float(prm & 0xFFFF0000u);
    }
    uint32_t w[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      // zero + scale * code: the product of 8 and 4 significant bits is exact in FP32.
      const float a = fmaf(scale, static_cast<float>((codes >> (8 * j)) & 15u), zero);
      const float b = fmaf(scale, static_cast<float>((codes >> (8 * j + 4)) & 15u), zero);
      const __nv_bfloat162 ab = __floats2bfloat162_rn(a, b);
      w[j] = *reinterpret_cast<const uint32_t*>(&ab);
    }
    uint16_t* y = (is_v ? p.V + token * p.ldv : p.K + token * p.ldk) + head * D + l * N;
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

unsigned grid_of(const Kv4Params& p, int sms) {
  const int64_t need = (p.tokens * p.heads + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(sms) * 8;
  return static_cast<unsigned>(need < cap ? need : cap);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Params& p, int d, bool vec, int sms, cudaStream_t s) {
  const dim3 g(grid_of(p, sms)), b(kThreads);
  if (d == 128)
    return vec ? launch_pdl(kv4_append_kernel<128, true>, g, b, 0, s, p)
               : launch_pdl(kv4_append_kernel<128, false>, g, b, 0, s, p);
  return vec ? launch_pdl(kv4_append_kernel<64, true>, g, b, 0, s, p)
             : launch_pdl(kv4_append_kernel<64, false>, g, b, 0, s, p);
}

cudaError_t launch_kv4_gather(const Kv4Params& p, int d, bool vec, int sms, cudaStream_t s) {
  const dim3 g(grid_of(p, sms)), b(kThreads);
  if (d == 128)
    return vec ? launch_pdl(kv4_gather_kernel<128, true>, g, b, 0, s, p)
               : launch_pdl(kv4_gather_kernel<128, false>, g, b, 0, s, p);
  return vec ? launch_pdl(kv4_gather_kernel<64, true>, g, b, 0, s, p)
             : launch_pdl(kv4_gather_kernel<64, false>, g, b, 0, s, p);
}

}  // namespace dg
