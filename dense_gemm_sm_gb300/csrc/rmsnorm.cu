// rmsnorm.cu -- residual addition and root-mean-square norm of a row, output BF16 or E4M3
// codes with one scale per row (what gemm_fp8_e4m3 reads):
//   h = x + r,  H = round(h),  y = (h * gain) * rstd,  rstd = 1 / sqrt(mean(h^2) + eps),
//   BF16:  Y = bf16(y)
//   E4M3:  amax = max |y|, scale = amax / 448, q = e4m3(y * (448 / amax)).
// h, the sum of squares and y are FP32; the norm is of the unrounded h, so the only roundings
// are the outputs' own.  rstd > 0 is one factor of the whole row and a product by it is
// monotone, so max |y| = max |h * gain| * rstd exactly: the maximum needs no pass after the
// norm and both reductions go together.
//
// HBM-bound: x and r are read once, H and Y written once.  A row stays in registers between
// the reduction and the output.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

struct None {};

__device__ __forceinline__ float bits_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bits_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint16_t pack_e4m3(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Eight consecutive elements, 16-byte accesses.
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  v[0] = bits_lo(u.x); v[1] = bits_hi(u.x); v[2] = bits_lo(u.y); v[3] = bits_hi(u.y);
  v[4] = bits_lo(u.z); v[5] = bits_hi(u.z); v[6] = bits_lo(u.w); v[7] = bits_hi(u.w);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                            pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[8]) {
  uint2 o;
  o.x = pack_e4m3(v[0], v[1]) | (static_cast<uint32_t>(pack_e4m3(v[2], v[3])) << 16);
  o.y = pack_e4m3(v[4], v[5]) | (static_cast<uint32_t>(pack_e4m3(v[6], v[7])) << 16);
  *reinterpret_cast<uint2*>(p) = o;
}
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16(v, 0.f)); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint8_t* p, float v) { *p = static_cast<uint8_t>(pack_e4m3(v, 0.f)); }

// Sum and maximum over the threads of one row: a warp, or the whole CTA.
__device__ __forceinline__ void row_reduce(float& sum, float& top, bool cta, float2* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (!cta) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) scratch[warp] = make_float2(sum, top);
  __syncthreads();
  const float2 v = lane < warps ? scratch[lane] : make_float2(0.f, 0.f);
  sum = v.x;
  top = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
}

// One row per 32 threads (8 rows a CTA) or per CTA of tpr threads, C chunks of 8 elements a
// thread.  VEC: chunk i of thread t is elements [8 (i tpr + t), + 8); otherwise a thread takes
// elements t, t + tpr, ... one by one, so that a warp's accesses stay contiguous.
template <typename XT, typename RT, typename YT, bool VEC, int C>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormParams p, const int tpr) {
  constexpr bool kRes = !std::is_same<RT, None>::value;
  constexpr bool kCodes = std::is_same<YT, uint8_t>::value;
  using R = typename std::conditional<kRes, RT, float>::type;
  __shared__ float2 scratch[32];
  pdl_trigger();
  pdl_wait();  // launched with programmatic serialisation: X may come from the previous kernel
  const bool cta = tpr > 32;
  const int t = cta ? threadIdx.x : (threadIdx.x & 31);
  const int64_t r = cta ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= p.rows) return;  // whole warps: a CTA of several rows has no barrier
  const XT* x = static_cast<const XT*>(p.X) + r * p.ldx;
  const R* res = kRes ? static_cast<const R*>(p.R) + r * p.ldr : nullptr;
  R* hout = kRes ? static_cast<R*>(p.H) + r * p.ldh : nullptr;
  YT* y = static_cast<YT*>(p.Y) + r * p.ldy;
  const int cols = static_cast<int>(p.cols);
  // An index of this thread's element j of chunk i.
  auto at = [&](int i, int j) { return VEC ? (i * tpr + t) * 8 + j : (8 * i + j) * tpr + t; };
  float h[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (VEC && at(i, 8) <= cols) {
      load8(x + at(i, 0), h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = at(i, j) < cols ? load1(x + at(i, j)) : 0.f;
    }
  }
  if (kRes) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[8];
      if (VEC && at(i, 8) <= cols) {
        load8(res + at(i, 0), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += v[j];
        store8(hout + at(i, 0), h[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at(i, j) < cols) {
            h[i][j] += load1(res + at(i, j));
            store1(hout + at(i, j), h[i][j]);
          }
      }
    }
  }
  // The gain multiplies at once: h itself is not needed again.
  float sum = 0.f, top = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float w[8];
    if (VEC && at(i, 8) <= cols) {
      load8(p.gain + at(i, 0), w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = at(i, j) < cols ? load1(p.gain + at(i, j)) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(h[i][j], h[i][j], sum);
      h[i][j] *= w[j];
      if (kCodes) top = fmaxf(top, fabsf(h[i][j]));
    }
  }
  row_reduce(sum, top, cta, scratch);
  float f = 1.f / sqrtf(sum / static_cast<float>(cols) + p.eps);
  float inv = 1.f;
  if (kCodes) {
    const float amax = top * f;
    inv = amax > 0.f ? __fdiv_rn(448.f, amax) : 0.f;
    if (t == 0) p.scales[r] = __fdiv_rn(amax, 448.f);
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = kCodes ? h[i][j] * f * inv : h[i][j] * f;
    if (VEC && at(i, 8) <= cols) {
      store8(y + at(i, 0), h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at(i, j) < cols) store1(y + at(i, j), h[i][j]);
    }
  }
}

// Rows too long for registers: one CTA a row, two passes, the second from L2.  H may be R, so
// the second pass reads each element of R before it writes that element of H.
template <typename XT, typename RT, typename YT>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(const NormParams p) {
  constexpr bool kRes = !std::is_same<RT, None>::value;
  constexpr bool kCodes = std::is_same<YT, uint8_t>::value;
  using R = typename std::conditional<kRes, RT, float>::type;
  __shared__ float2 scratch[32];
  pdl_trigger();
  pdl_wait();
  const int64_t r = blockIdx.x;
  const XT* x = static_cast<const XT*>(p.X) + r * p.ldx;
  const R* res = kRes ? static_cast<const R*>(p.R) + r * p.ldr : nullptr;
  R* hout = kRes ? static_cast<R*>(p.H) + r * p.ldh : nullptr;
  YT* y = static_cast<YT*>(p.Y) + r * p.ldy;
  float sum = 0.f, top = 0.f;
#pragma unroll 4
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float h = load1(x + c) + (kRes ? load1(res + c) : 0.f);
    sum = fmaf(h, h, sum);
    if (kCodes) top = fmaxf(top, fabsf(h * load1(p.gain + c)));
  }
  row_reduce(sum, top, true, scratch);
  const float f = 1.f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
  float inv = 1.f;
  if (kCodes) {
    const float amax = top * f;
    inv = amax > 0.f ? __fdiv_rn(448.f, amax) : 0.f;
    if (threadIdx.x == 0) p.scales[r] = __fdiv_rn(amax, 448.f);
  }
#pragma unroll 4
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float h = load1(x + c) + (kRes ? load1(res + c) : 0.f);
    if (kRes) store1(hout + c, h);
    const float v = h * load1(p.gain + c) * f;
    store1(y + c, kCodes ? v * inv : v);
  }
}

template <typename XT, typename RT, typename YT>
cudaError_t launch_typed(const NormParams& p, bool vec, cudaStream_t s) {
  const int64_t chunks = (p.cols + 7) / 8;
  // Chunks a thread: 1 for as long as a CTA holds the row (16384 x 4096 with an FP32 residual:
  // 107 us, 118 with 2, 124 with 4), except that rows of up to 512 elements then fit a warp with
  // 2 (16384 x 512: 17.3 us in CTAs of 64 threads, 13.8 so); over 8192 elements 4 (2048 x 16384:
  // 58 us, 65 with 2).  Unaligned rows over 8192 elements take the two-pass kernel: an element at
  // a time, more than 8 do not stay in registers.
  if (chunks > (vec ? 4 : 1) * 1024)
    return launch_pdl(rmsnorm_long_kernel<XT, RT, YT>, dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, s, p);
  const int c = !vec ? 1 : chunks > 1024 ? 4 : chunks > 32 && chunks <= 64 ? 2 : 1;
  int tpr = static_cast<int>((chunks + c - 1) / c);
  tpr = (tpr + 31) / 32 * 32;
  const int rows_per_cta = tpr == 32 ? 8 : 1;
  const dim3 grid(static_cast<unsigned>((p.rows + rows_per_cta - 1) / rows_per_cta)), block(tpr * rows_per_cta);
  if (vec)
    return c == 1   ? launch_pdl(rmsnorm_kernel<XT, RT, YT, true, 1>, grid, block, 0, s, p, tpr)
           : c == 2 ? launch_pdl(rmsnorm_kernel<XT, RT, YT, true, 2>, grid, block, 0, s, p, tpr)
                    : launch_pdl(rmsnorm_kernel<XT, RT, YT, true, 4>, grid, block, 0, s, p, tpr);
  return launch_pdl(rmsnorm_kernel<XT, RT, YT, false, 1>, grid, block, 0, s, p, tpr);
}

template <typename XT, typename RT>
cudaError_t launch_out(const NormParams& p, bool vec, cudaStream_t s) {
  return p.scales ? launch_typed<XT, RT, uint8_t>(p, vec, s) : launch_typed<XT, RT, uint16_t>(p, vec, s);
}

template <typename XT>
cudaError_t launch_res(const NormParams& p, bool r_f32, bool vec, cudaStream_t s) {
  if (!p.R) return launch_out<XT, None>(p, vec, s);
  return r_f32 ? launch_out<XT, float>(p, vec, s) : launch_out<XT, uint16_t>(p, vec, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormParams& p, bool x_f32, bool r_f32, bool vec, int sms,
                           cudaStream_t s) {
  (void)sms;
  return x_f32 ? launch_res<float>(p, r_f32, vec, s) : launch_res<uint16_t>(p, r_f32, vec, s);
}

}  // namespace dg
