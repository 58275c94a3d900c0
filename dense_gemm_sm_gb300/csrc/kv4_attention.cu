// kv4_attention.cu -- attention of the newest tokens of each sequence over the paged 4-bit
// cache: for query i of sequence b (its position is len_b - Lq + i),
//   O = sum_j softmax_j(scale * q . K_j) V_j   over the keys j <= len_b - Lq + i,
// K_j and V_j being the values the cache's codes stand for.  A query that sees no key gets 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

constexpr int kThreads = 256;

// One CTA per (sequence, query, query head): a warp takes every eighth key, the lanes share
// its d elements, and the warps' running maxima, sums and outputs are joined at the end.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_attention_kernel(const Kv4AttnParams p) {
  constexpr int N = D / 32;
  pdl_trigger();
  pdl_wait();
  const int heads_q = p.heads * p.group;
  const int64_t id = blockIdx.x;
  const int hq = static_cast<int>(id % heads_q);
  const int64_t i = id / heads_q % p.Lq, b = id / heads_q / p.Lq;
  const int head = hq / p.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t len = p.lens[b];
  const int64_t cap = p.ldt * p.page_size;
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0) atomicCAS(p.index_word, 0u, kDevBadIndex);
    len = len < 0 ? 0 : cap;
  }
  const int64_t keys = len - p.Lq + i + 1;
  const uint16_t* q = p.Q + b * p.strideQ + i * p.ldq + hq * D + lane * N;
  float qv[N], acc[N], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    qv[j] = __uint_as_float(static_cast<uint32_t>(q[j]) << 16);
    acc[j] = 0.f;
  }
  for (int64_t k = warp; k < keys; k += kThreads / 32) {
    const int32_t page = p.table[b * p.ldt + k / p.page_size];
    if (page < 0 || page >= p.pages) {
      if (lane == 0) atomicCAS(p.index_word, 0u, kDevBadIndex);
      continue;
    }
    const int in = static_cast<int>(k % p.page_size), u = in & 15;
    const uint8_t* rec = p.data + ((static_cast<int64_t>(page) * p.heads + head) * (p.page_size / 16) + (in >> 4)) *
                                      kv4_record_bytes(D);
    const uint32_t kp = *reinterpret_cast<const uint32_t*>(rec + 16 * D + u * 4);
    const uint32_t vp = *reinterpret_cast<const uint32_t*>(rec + 16 * D + 64 + u * 4);
    const float ks = __uint_as_float(kp << 16), kz = __uint_as_float(kp & 0xFFFF0000u);
    const float vs = __uint_as_float(vp << 16), vz = __uint_as_float(vp & 0xFFFF0000u);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = lane * N + j;
      const uint32_t code = (rec[u * (D / 2) + c / 2] >> (4 * (c & 1))) & 15u;
      dot = fmaf(qv[j], fmaf(ks, static_cast<float>(code), kz), dot);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float s = dot * p.c_log2;
    const float mn = fmaxf(m, s), r = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * r + w;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = lane * N + j, g = c / (D / 8), cl = c % (D / 8);
      const uint8_t byte = rec[8 * D + (((u >> 3) * 8 + g) * 4 + ((u & 7) >> 1)) * (D / 8) + cl / 4 * 4 +
                               (u & 1) * 2 + (cl & 3) / 2];
      const uint32_t code = (byte >> (4 * (c & 1))) & 15u;
      acc[j] = fmaf(w, fmaf(vs, static_cast<float>(code), vz), acc[j] * r);
    }
  }
  __shared__ float sm[8], sl[8], sa[8][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) sa[warp][lane * N + j] = acc[j];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float top = -INFINITY, tl = 0.f, ta = 0.f;
    for (int w = 0; w < 8; ++w) top = fmaxf(top, sm[w]);
    for (int w = 0; w < 8; ++w) {
      const float r = sm[w] > -INFINITY ? exp2f(sm[w] - top) : 0.f;
      tl += sl[w] * r;
      ta += sa[w][c] * r;
    }
    const __nv_bfloat16 o = __float2bfloat16_rn(tl > 0.f ? ta / tl : 0.f);
    p.O[b * p.strideO + i * p.ldo + hq * D + c] = __bfloat16_as_ushort(o);
  }
}

}  // namespace

int64_t kv4_attention_ws_bytes(int64_t batch, int64_t Lq, int64_t heads_q, int64_t heads_kv, int d) {
  (void)batch; (void)Lq; (void)heads_q; (void)heads_kv; (void)d;
  return 16;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, int d, int sms, cudaStream_t s) {
  (void)sms;
  const dim3 g(static_cast<unsigned>(p.batch * p.Lq * p.heads * p.group)), b(kThreads);
  return d == 128 ? launch_pdl(kv4_attention_kernel<128>, g, b, 0, s, p)
                  : launch_pdl(kv4_attention_kernel<64>, g, b, 0, s, p);
}

}  // namespace dg
