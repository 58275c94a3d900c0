// moe.cu -- a mixture-of-experts layer for few tokens, from the router's logits on:
//   p = softmax(logits) over the E experts; the `top` largest logits are chosen (ties: the
//   lowest expert), w = p (over the sum of the chosen p when renorm);
//   z = bf16(SiLU(x W_g[e]) * (x W_u[e])),  y = bf16(sum_e w_e (z W_d[e])).
// Products are BF16 with FP32 sums; z is rounded once, as an operand of the second product.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

struct Layout {
  int64_t ids, weights, z, total;
};
constexpr int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
Layout layout_of(int64_t T, int64_t I, int64_t top) {
  Layout l;
  l.ids = 0;
  l.weights = up16(T * top * 4);
  l.z = 2 * l.weights;
  l.total = l.z + up16(T * top * I * 2);
  return l;
}

// One warp per token: the chosen experts in order of their logits.
__global__ void moe_route_kernel(const MoeParams p, int32_t* ids, float* weights) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x;
  const float* row = p.logits + static_cast<int64_t>(blockIdx.x) * p.ldl;
  float top = -INFINITY, sum = 0.f;
  for (int e = lane; e < p.E; e += 32) top = fmaxf(top, row[e]);
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  for (int e = lane; e < p.E; e += 32) sum += row[e] > -INFINITY ? expf(row[e] - top) : 0.f;
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  float last = INFINITY, chosen = 0.f;
  int last_e = -1;
  for (int k = 0; k < p.top; ++k) {
    float best = -INFINITY;
    int be = 0x7FFFFFFF;
    for (int e = lane; e < p.E; e += 32) {
      const float v = row[e];
      const bool after = v < last || (v == last && e > last_e);
      if (after && (v > best || (v == best && e < be))) {
        best = v;
        be = e;
      }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(~0u, best, o);
      const int oe = __shfl_xor_sync(~0u, be, o);
      if (ov > best || (ov == best && oe < be)) {
        best = ov;
        be = oe;
      }
    }
    const bool real = best > -INFINITY;
    const float w = real ? expf(best - top) : 0.f;
    chosen += w;
    if (lane == 0) {
      ids[static_cast<int64_t>(blockIdx.x) * p.top + k] = real ? be : -1;
      weights[static_cast<int64_t>(blockIdx.x) * p.top + k] = w;
    }
    last = best;
    last_e = be;
  }
  const float by = p.renorm ? chosen : sum;
  __syncwarp();
  for (int k = lane; k < p.top; k += 32) {
    float& w = weights[static_cast<int64_t>(blockIdx.x) * p.top + k];
    w = by > 0.f ? w / by : 0.f;
  }
}

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__global__ void moe_up_kernel(const MoeParams p, const int32_t* ids, uint16_t* z) {
  const int64_t pair = blockIdx.y, n = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int e = ids[pair];
  if (e < 0 || n >= p.I) return;
  const uint16_t* x = p.X + pair / p.top * p.ldx;
  const uint16_t* wg = p.Wg + e * p.strideWg + n;
  const uint16_t* wu = p.Wu + e * p.strideWu + n;
  float g = 0.f, u = 0.f;
  for (int64_t k = 0; k < p.K; ++k) {
    const float xv = bf(x[k]);
    g = fmaf(xv, bf(wg[k * p.ldwg]), g);
    u = fmaf(xv, bf(wu[k * p.ldwu]), u);
  }
  z[pair * p.I + n] = __bfloat16_as_ushort(__float2bfloat16_rn(g / (1.f + expf(-g)) * u));
}

__global__ void moe_down_kernel(const MoeParams p, const int32_t* ids, const float* weights, const uint16_t* z) {
  const int64_t t = blockIdx.y, n = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (n >= p.K) return;
  float y = 0.f;
  for (int k = 0; k < p.top; ++k) {
    const int64_t pair = t * p.top + k;
    const int e = ids[pair];
    if (e < 0) continue;
    const uint16_t* wd = p.Wd + e * p.strideWd + n;
    float s = 0.f;
    for (int64_t i = 0; i < p.I; ++i) s = fmaf(bf(z[pair * p.I + i]), bf(wd[i * p.ldwd]), s);
    y = fmaf(weights[pair], s, y);
  }
  p.Y[t * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

}  // namespace

int64_t moe_ws_bytes(int64_t T, int64_t K, int64_t I, int64_t E, int64_t top) {
  (void)K; (void)E;
  return layout_of(T, I, top).total;
}

cudaError_t launch_moe(const MoeParams& p, int sms, cudaStream_t s) {
  (void)sms;
  const Layout l = layout_of(p.T, p.I, p.top);
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  int32_t* ids = reinterpret_cast<int32_t*>(ws + l.ids);
  float* weights = reinterpret_cast<float*>(ws + l.weights);
  uint16_t* z = reinterpret_cast<uint16_t*>(ws + l.z);
  cudaError_t e = launch_pdl(moe_route_kernel, dim3(static_cast<unsigned>(p.T)), dim3(32), 0, s, p, ids, weights);
  if (e != cudaSuccess) return e;
  const unsigned pairs = static_cast<unsigned>(p.T * p.top);
  moe_up_kernel<<<dim3(static_cast<unsigned>((p.I + 127) / 128), pairs), 128, 0, s>>>(p, ids, z);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  moe_down_kernel<<<dim3(static_cast<unsigned>((p.K + 127) / 128), static_cast<unsigned>(p.T)), 128, 0, s>>>(p, ids, weights, z);
  return cudaGetLastError();
}

}  // namespace dg
