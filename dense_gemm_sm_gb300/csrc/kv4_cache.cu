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
// takes one token and a run of its heads, four at a time with their loads together: lanes 0-15
// the key's row, lanes 16-31 the value's, d / 16 elements a lane (16-byte accesses at d = 128).
// What a token needs once (its slot's page) is found once, and quotients come from a reciprocal,
// with the division itself only where its rounding could decide: a warp per (token, head) with
// 64-bit indices and true divisions issued 450 instructions for each and took 25 us for 8192
// tokens of 8 heads, which are 6 us of HBM traffic.
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
        float v[N];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          v[2 * j] = __uint_as_float(w[x][j] << 16);
          v[2 * j + 1] = __uint_as_float(w[x][j] & 0xFFFF0000u);
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
        // round(difference / scale), halves to even: n from the product by the reciprocal is the
        // quotient's nearest integer or, next to a half, its neighbour.  The remainder d - n scale
        // is exact, so t = 2 |remainder| - scale tells: positive, n is the wrong neighbour; zero,
        // a half, where n has to be even.  (A quotient that is no half is never rounded to one:
        // it differs by more than half an FP32 step, as d and scale have 24 and 8 bits.)  Halves
        // are common, differences of BF16 values over a BF16 scale.
        const float inv = __frcp_rn(scale);
        constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
        float n[N], rem[N], worst = -1.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float d = __fsub_rn(v[j], lo);
          n[j] = fmaf(d, inv, kRound) - kRound;
          rem[j] = fmaf(-n[j], scale, d);
          worst = fmaxf(worst, fmaf(2.f, fabsf(rem[j]), -scale));
        }
        uint32_t codes = 0;
        if (!(scale >= 7.5e-37f)) {  // the reciprocal could overflow: the division itself
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float q = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(v[j], lo), scale)) : 0.f;
            codes |= static_cast<uint32_t>(fminf(fmaxf(q, 0.f), 15.f)) << (4 * j);
          }
        } else {
          if (worst >= 0.f) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
              const float t = fmaf(2.f, fabsf(rem[j]), -scale);
              const bool odd = __float_as_uint(n[j] + kRound) & 1u;
              if (t > 0.f || (t == 0.f && odd)) n[j] += rem[j] > 0.f ? 1.f : -1.f;
            }
          }
#pragma unroll
          for (int j = 0; j < N; ++j)
            codes |= (__float_as_uint(fminf(n[j], 15.f) + kRound) & 15u) << (4 * j);
        }
        uint8_t* rec = rec0 + (h + x) * stride;
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
    for (int h = h0; h < h1; h += H) {
      uint32_t codes[H], prm[H];
#pragma unroll
      for (int x = 0; x < H; ++x) {
        codes[x] = prm[x] = 0;  // the value 0
        if (!have) continue;
        const uint8_t* rec = rec0 + (h + x) * stride;
        if (!is_v) {
          if (N == 8) codes[x] = *reinterpret_cast<const uint32_t*>(rec + u * (D / 2) + l * 4);
          else codes[x] = *reinterpret_cast<const uint16_t*>(rec + u * (D / 2) + l * 2);
        } else {
#pragma unroll
          for (int j = 0; j < N / 4; ++j)
            codes[x] |= static_cast<uint32_t>(
                            *reinterpret_cast<const uint16_t*>(rec + 8 * D + v_piece<D>(u, l * (N / 4) + j)))
                        << (16 * j);
        }
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
Shape shape_of(const Kv4Params& p, int sms) {
  const int64_t slots = static_cast<int64_t>(sms) * 64;  // resident warps
  int64_t runs = slots / (p.tokens < slots ? p.tokens : slots);
  if (runs > p.heads) runs = p.heads;
  Shape s;
  s.heads_per_warp = static_cast<int>((p.heads + runs - 1) / runs);
  s.in_flight = p.heads % 4 == 0 && s.heads_per_warp >= 4 ? 4 : 1;
  if (s.in_flight == 4) s.heads_per_warp = (s.heads_per_warp + 3) / 4 * 4;
  const int64_t need = (p.tokens + kThreads / 32 - 1) / (kThreads / 32), cap = static_cast<int64_t>(sms) * 8;
  s.grid = dim3(static_cast<unsigned>(need < cap ? need : cap),
                static_cast<unsigned>((p.heads + s.heads_per_warp - 1) / s.heads_per_warp));
  return s;
}

}  // namespace

#define DG_KV4_LAUNCH(KERNEL, D, VEC)                                                              \
  (f.in_flight == 4 ? launch_pdl(KERNEL<D, VEC, 4>, f.grid, b, 0, s, p, f.heads_per_warp)        \
                    : launch_pdl(KERNEL<D, VEC, 1>, f.grid, b, 0, s, p, f.heads_per_warp))

cudaError_t launch_kv4_append(const Kv4Params& p, int d, bool vec, int sms, cudaStream_t s) {
  const Shape f = shape_of(p, sms);
  const dim3 b(kThreads);
  if (d == 128) return vec ? DG_KV4_LAUNCH(kv4_append_kernel, 128, true) : DG_KV4_LAUNCH(kv4_append_kernel, 128, false);
  return vec ? DG_KV4_LAUNCH(kv4_append_kernel, 64, true) : DG_KV4_LAUNCH(kv4_append_kernel, 64, false);
}

cudaError_t launch_kv4_gather(const Kv4Params& p, int d, bool vec, int sms, cudaStream_t s) {
  const Shape f = shape_of(p, sms);
  const dim3 b(kThreads);
  if (d == 128) return vec ? DG_KV4_LAUNCH(kv4_gather_kernel, 128, true) : DG_KV4_LAUNCH(kv4_gather_kernel, 128, false);
  return vec ? DG_KV4_LAUNCH(kv4_gather_kernel, 64, true) : DG_KV4_LAUNCH(kv4_gather_kernel, 64, false);
}
#undef DG_KV4_LAUNCH

}  // namespace dg
