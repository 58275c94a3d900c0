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
// The same from any address: the 16-byte words that hold them, and a shift that is one of the
// whole row, so no lane goes its own way.
__device__ __forceinline__ void load8_any(const uint16_t* p, float (&v)[8]) {
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / 2;
  const uint4* g = reinterpret_cast<const uint4*>(p - shift);
  const uint4 a = g[0];
  uint32_t w[7] = {a.x, a.y, a.z, a.w, 0, 0, 0};
  if (shift != 0) {
    const uint4 b = g[1];
    if (shift & 4) {
      w[0] = a.z; w[1] = a.w; w[2] = b.x; w[3] = b.y; w[4] = b.z; w[5] = b.w;
    } else {
      w[4] = b.x; w[5] = b.y; w[6] = b.z;
    }
    if (shift & 2) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (shift & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __byte_perm(w[i], w[i + 1], 0x5432);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bits_lo(w[i]);
    v[2 * i + 1] = bits_hi(w[i]);
  }
}
__device__ __forceinline__ void load8_any(const float* p, float (&v)[8]) {
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / 4;
  const float4* g = reinterpret_cast<const float4*>(p - shift);
  const float4 a = g[0], b = g[1];
  float w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, 0.f, 0.f, 0.f, 0.f};
  if (shift != 0) {
    const float4 c = g[2];
    w[8] = c.x; w[9] = c.y; w[10] = c.z; w[11] = c.w;
    if (shift & 2) {
#pragma unroll
      for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
    }
    if (shift & 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = w[i + 1];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = w[i];
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

// Sum and maximum over the threads of one row: `lanes` of a warp, or the whole CTA.
__device__ __forceinline__ void row_reduce(float& sum, float& top, int lanes, bool cta, float2* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= lanes) continue;
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

// The largest output amax, and what makes codes of h * gain, from top = max |h * gain|: f becomes
// the first factor, inv the second.  The ends of the range stand in one branch (1024 x 4096 from L2:
// 5.8 us with a choice for each among the ordinary rows' operations, 5.65 so, 5.55 without them).
__device__ __forceinline__ float code_factors(float top, float& f, float& inv) {
  const float amax = top * f;
  if (amax >= 1e-35f) {
    inv = __fdiv_rn(448.f, amax);
    return amax;
  }
  inv = 0.f;
  if (amax > 0.f) {
    // 448 / amax may pass FP32's range, and codes be +-448 and NaN: they are taken as (h * gain) *
    // (448 / top), which is the same, where need be with 2^64 between the two.
    f = top < 1.f ? 0x1p64f : 1.f;
    inv = __fdiv_rn(448.f, top * f);
    return amax;
  }
  if (top == 0.f && f > 0.f) return f = 0.f;  // zeros; f is 1 / 0 when eps is 0
  return amax;
}

// One row per CTA of tpr threads, per warp (8 rows a CTA) or, PART, per tpr = 8 or 16 lanes, C
// chunks of 8 elements a thread (200000 rows of 128: 19 us, 48 in warps half of which idle; 64 wide
// with a residual and codes 16 and 74).
//   kAligned: chunk i of thread t is elements [8 (i tpr + t), + 8);
//   kShifted: rows begin anywhere, but those of H as far from an aligned address as those of Y:
//     chunks are the aligned ones of Y, what is read comes from any address; chunks within 8
//     elements of the row's ends go one element at a time, so that nothing outside is read;
//   kSingle: a thread takes elements t, t + tpr, ... one by one, so that a warp's accesses stay
//     contiguous.
enum Mode { kSingle, kAligned, kShifted };
// (Two CTAs an SM cost the shifted form a few spills: 8192 x 4096, FP32 residual, codes, 99 -> 84 us.)
template <typename XT, typename RT, typename YT, Mode M, int C, bool PART = false>
__global__ void __launch_bounds__(1024, M == kShifted && C == 1 ? 2 : 0) rmsnorm_kernel(const NormParams p, const int tpr) {
  constexpr bool kRes = !std::is_same<RT, None>::value;
  constexpr bool kCodes = std::is_same<YT, uint8_t>::value;
  using R = typename std::conditional<kRes, RT, float>::type;
  __shared__ float2 scratch[32];
  pdl_trigger();
  pdl_wait();  // launched with programmatic serialisation: X may come from the previous kernel
  const bool cta = !PART && tpr > 32;
  const int t = cta ? threadIdx.x : (threadIdx.x & (PART ? tpr - 1 : 31)), shift = PART && tpr == 8 ? 3 : PART ? 4 : 5;
  const int64_t r = cta ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (blockDim.x >> shift) + (threadIdx.x >> shift);
  // A CTA of several rows has no barrier, so whole warps can go; part of one past the last row
  // stays for the others' sums.
  const bool live = r < p.rows;
  if (!PART && !live) return;
  const XT* x = static_cast<const XT*>(p.X) + r * p.ldx;
  const R* res = kRes ? static_cast<const R*>(p.R) + r * p.ldr : nullptr;
  R* hout = kRes ? static_cast<R*>(p.H) + r * p.ldh : nullptr;
  YT* y = static_cast<YT*>(p.Y) + r * p.ldy;
  const int cols = !PART || live ? static_cast<int>(p.cols) : 0;
  const int skip = M == kShifted ? static_cast<int>(reinterpret_cast<uintptr_t>(y) / sizeof(YT) & 7) : 0;
  // An index of this thread's element j of chunk i.
  auto at = [&](int i, int j) { return M == kSingle ? (8 * i + j) * tpr + t : (i * tpr + t) * 8 + j - skip; };
  auto inside = [&](int i, int j) { return (M != kShifted || at(i, j) >= 0) && at(i, j) < cols; };
  auto whole = [&](int i) {
    return M == kAligned ? at(i, 8) <= cols : M == kShifted && at(i, 0) >= 8 && at(i, 16) <= cols;
  };
  auto load = [&](const auto* from, float (&v)[8]) {
    if constexpr (M == kShifted) load8_any(from, v);
    else load8(from, v);
  };
  float h[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if (whole(i)) {
      load(x + at(i, 0), h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = inside(i, j) ? load1(x + at(i, j)) : 0.f;
    }
  }
  if (kRes) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float v[8];
      if (whole(i)) {
        load(res + at(i, 0), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += v[j];
        store8(hout + at(i, 0), h[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (inside(i, j)) {
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
    if (whole(i)) {
      load(p.gain + at(i, 0), w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = inside(i, j) ? load1(p.gain + at(i, j)) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(h[i][j], h[i][j], sum);
      h[i][j] *= w[j];
      if (kCodes) top = fmaxf(top, fabsf(h[i][j]));
    }
  }
  row_reduce(sum, top, PART ? tpr : 32, cta, scratch);
  float f = 1.f / sqrtf(sum / static_cast<float>(static_cast<int>(p.cols)) + p.eps);
  float inv = 1.f;
  if (kCodes) {
    const float amax = code_factors(top, f, inv);
    if (t == 0 && (!PART || live)) p.scales[r] = __fdiv_rn(amax, 448.f);
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = kCodes ? h[i][j] * f * inv : h[i][j] * f;
    if (whole(i)) {
      store8(y + at(i, 0), h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (inside(i, j)) store1(y + at(i, j), h[i][j]);
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
  row_reduce(sum, top, 32, true, scratch);
  float f = 1.f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
  float inv = 1.f;
  if (kCodes) {
    const float amax = code_factors(top, f, inv);
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
cudaError_t launch_typed(const NormParams& p, Mode m, cudaStream_t s) {
  // Shifted chunks pay from 128 elements a row (16384 rows of 100, 200, 1000 BF16: 9.3, 10.3, 29 us,
  // one at a time 8.7, 14.7, 69).  FP32 elements fill a warp's accesses one at a time too: few
  // short rows are faster so (1000 x 777: 3.3 us and 3.5; with a residual and codes 4.8 and 6.4;
  // 16384 x 777: 26 and 19.5; 1000 x 2777: 7.6 and 5.6).
  constexpr bool kWide = std::is_same<XT, float>::value || std::is_same<RT, float>::value;
  const int64_t least = kWide && p.rows * p.cols < (int64_t{1} << 22) ? 1024 : 128;
  if (m == kShifted && p.cols < least) m = kSingle;
  const int64_t chunks = (p.cols + (m == kShifted ? 14 : 7)) / 8;
  // Chunks a thread: 1 for as long as a CTA holds the row (16384 x 4096 with an FP32 residual:
  // 107 us, 118 with 2, 124 with 4), except that rows of up to 512 elements then fit a warp with
  // 2 (16384 x 512: 17.3 us in CTAs of 64 threads, 13.8 so); over 8192 elements 3 or 4
  // (2048 x 16384: 58 us with 4, 65 with 2): what leaves more CTAs of 64 registers a thread to an SM,
  // and 3 where both leave the same (4096 x 12288, residual, codes: 84 us with 3, 99 with 4; 4096 x
  // 10240 81 and 72); shifted 2 (4096 x 8190: 82 us, one element at a time 191).  Longer rows,
  // and those over 8192 elements that go one at a time, take the two-pass kernel: they do not stay
  // in registers (2048 x 16384 shifted, 4 chunks: 116 us, in two passes 80).
  if (chunks > (m == kSingle ? 1 : m == kShifted ? 2 : 4) * 1024)
    return launch_pdl(rmsnorm_long_kernel<XT, RT, YT>, dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, s, p);
  auto threads = [&](int64_t each) { return ((chunks + each - 1) / each + 31) / 32 * 32; };
  const bool three = threads(3) <= 1024 && 1024 / threads(3) == 1024 / threads(4);
  const int c = chunks > 1024 ? (m == kShifted ? 2 : three ? 3 : 4) : m == kAligned && chunks > 32 && chunks <= 64 ? 2 : 1;
  int tpr = static_cast<int>((chunks + c - 1) / c);
  tpr = tpr <= 8 ? 8 : tpr <= 16 ? 16 : (tpr + 31) / 32 * 32;
  const int rows_per_cta = tpr <= 32 ? 256 / tpr : 1;
  const dim3 grid(static_cast<unsigned>((p.rows + rows_per_cta - 1) / rows_per_cta)), block(tpr * rows_per_cta);
  if (tpr < 32)  // (the shifted form begins with longer rows)
    return m == kAligned ? launch_pdl(rmsnorm_kernel<XT, RT, YT, kAligned, 1, true>, grid, block, 0, s, p, tpr)
                         : launch_pdl(rmsnorm_kernel<XT, RT, YT, kSingle, 1, true>, grid, block, 0, s, p, tpr);
  if (m == kAligned)
    return c == 1   ? launch_pdl(rmsnorm_kernel<XT, RT, YT, kAligned, 1>, grid, block, 0, s, p, tpr)
           : c == 2 ? launch_pdl(rmsnorm_kernel<XT, RT, YT, kAligned, 2>, grid, block, 0, s, p, tpr)
           : c == 3 ? launch_pdl(rmsnorm_kernel<XT, RT, YT, kAligned, 3>, grid, block, 0, s, p, tpr)
                    : launch_pdl(rmsnorm_kernel<XT, RT, YT, kAligned, 4>, grid, block, 0, s, p, tpr);
  if (m == kShifted)
    return c == 1 ? launch_pdl(rmsnorm_kernel<XT, RT, YT, kShifted, 1>, grid, block, 0, s, p, tpr)
                  : launch_pdl(rmsnorm_kernel<XT, RT, YT, kShifted, 2>, grid, block, 0, s, p, tpr);
  return launch_pdl(rmsnorm_kernel<XT, RT, YT, kSingle, 1>, grid, block, 0, s, p, tpr);
}

template <typename XT, typename RT>
cudaError_t launch_out(const NormParams& p, Mode m, cudaStream_t s) {
  return p.scales ? launch_typed<XT, RT, uint8_t>(p, m, s) : launch_typed<XT, RT, uint16_t>(p, m, s);
}

template <typename XT>
cudaError_t launch_res(const NormParams& p, bool r_f32, Mode m, cudaStream_t s) {
  if (!p.R) return launch_out<XT, None>(p, m, s);
  return r_f32 ? launch_out<XT, float>(p, m, s) : launch_out<XT, uint16_t>(p, m, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormParams& p, bool x_f32, bool r_f32, bool vec, cudaStream_t s) {
  // Where rows of H and of Y are equally far from an aligned address.
  const uint64_t y = reinterpret_cast<uintptr_t>(p.Y) / (p.scales ? 1 : 2), h = reinterpret_cast<uintptr_t>(p.H) / (r_f32 ? 4 : 2);
  const uint64_t period = r_f32 ? 4 : 8;  // elements of 16 bytes of H
  const bool together = !p.R || ((h - y) % period == 0 && (p.rows == 1 || static_cast<uint64_t>(p.ldh - p.ldy) % period == 0));
  const Mode m = vec ? kAligned : together ? kShifted : kSingle;
  return x_f32 ? launch_res<float>(p, r_f32, m, s) : launch_res<uint16_t>(p, r_f32, m, s);
}

}  // namespace dg
