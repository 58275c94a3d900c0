// moe.cu -- a mixture-of-experts layer for few tokens, from the router's logits on:
//   p = softmax(logits) over the E experts; the `top` largest logits are chosen (ties: the
//   lowest expert), w = p (over the sum of the chosen p when renorm);
//   z = bf16(SiLU(x W_g[e]) * (x W_u[e])),  y = bf16(sum_e w_e (z W_d[e])).
// Products are BF16 with FP32 sums; z is rounded once, as an operand of the second product.
//
// With at most 64 tokens every weight of a chosen expert is used a few times: reading each
// once from HBM bounds the layer.  Two kernels, one CTA per SM each, the second launched
// programmatically behind the first:
//   * up: every CTA routes all tokens itself (a warp per token; less than a launch costs), then
//     the work of the active experts -- (expert, 64 columns of W_g and of W_u, 64 rows of K)
//     units -- is cut evenly over the CTAs, whatever the experts' number;
//   * down: (128 columns of W_d, expert, 64 rows of I) units, cut the same way.  A column tile
//     sums over experts in FP32 in shared memory, one addition per expert and token.
// Units stream through a ring of TMA stages into tcgen05 with the weights as the 128-row
// operand (as they lie, N contiguous) and the tokens as the narrow one: all T tokens in the
// first product (rows of other experts are ignored: gathering them would cost more than their
// columns), an expert's own rows, 16 at a time, in the second, whose input the first writes
// sorted by expert.  A tile cut between CTAs is finished by the last of them to arrive, which
// adds the parts in CTA order: results do not depend on arrival.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg_internal.h"
#include "ptx.cuh"
#include "serving.h"

namespace dg {
namespace {

constexpr int kMaxCtas = 160;        // CTAs that the workspace has room for
constexpr int kMaxT = 64, kMaxE = 512, kMaxTop = 16, kMaxPairs = kMaxT * kMaxTop;
constexpr int BK = 64;               // rows of a unit
constexpr uint32_t W_BYTES = 128 * BK * 2;
constexpr int kUpThreads = 512;      // routing: a warp per token
constexpr int kDownThreads = 192;
constexpr int kPrefetch = 10;        // units of W_d that the up kernel asks L2 for, per CTA

// What the up kernel tells the down kernel.
struct Routes {
  int32_t active;                    // experts with at least one token
  int32_t expert[kMaxE];             // in ascending order
  int32_t off[kMaxE + 1];            // their first rows of Z
  int32_t token[kMaxPairs];          // of a row of Z
  float weight[kMaxPairs];
};

// Workspace: counters (zero between calls), routes, Z, parts of cut tiles.
constexpr int64_t kCounters = 2 * kMaxCtas;
constexpr int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
constexpr int64_t kRoutesAt = up256(kCounters * 4);
constexpr int64_t kPartsAt = kRoutesAt + up256(sizeof(Routes));
constexpr int ntok_of(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }
constexpr int64_t part_floats(int64_t T) { return ntok_of(T) * 128; }
constexpr int64_t z_at(int64_t T) { return kPartsAt + 2 * kMaxCtas * part_floats(T) * 4; }
constexpr int64_t ldz_of(int64_t I) { return (I + 7) / 8 * 8; }

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

__device__ __forceinline__ uint32_t take_ticket(uint32_t* a) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a) : "memory");
  return old;
}
// Orders this thread's view of ordinary global stores before its TMA loads.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l2_3d(const CUtensorMap* map, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

struct Maps {
  CUtensorMap a, a2, b;  // up: W_g, W_u, X; down: W_d, -, Z
};

template <int STAGES>
struct Pipe {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem_base, abort, is_last, seg_ok;
  __device__ void init() {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 4);
    }
    mbar_init(smem_u32(&drain), 1);
    abort = 0;
    is_last = 0;
    seg_ok = 0;
    fence_barrier_init();
  }
  // After a producer gave up: its copies in flight end before the CTA does.
  __device__ void drain_loads(uint32_t it, uint32_t* status) {
    uint32_t never = 0;
    for (uint32_t j = it > STAGES ? it - STAGES : 0u; j < it; ++j)
      mbar_wait(smem_u32(&full[j % STAGES]), (j / STAGES) & 1u, &never, status, kDevTimeoutDrain);
  }
};

template <int NTOK>
struct Cfg {
  static constexpr int kStages = NTOK == 64 ? 7 : 8;
  static constexpr uint32_t kX = NTOK * BK * 2;
  static constexpr uint32_t kRing = kStages * (W_BYTES + kX);
  static constexpr uint32_t kTmem = NTOK == 16 ? 32 : 2 * NTOK;
  static constexpr int kHalf = NTOK < 32 ? NTOK : 32;  // tokens in registers at a time
};

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  uint32_t r[N];
  if constexpr (N == 16) tmem_ld_32x32b_x16(taddr, r);
  else tmem_ld_32x32b_x32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int t = 0; t < N; ++t) v[t] = __uint_as_float(r[t]);
}

// ------------------------------------------------------------------ routing
struct RouteShared {
  uint32_t mask[kMaxE][2];             // tokens of an expert
  int32_t id[kMaxT][kMaxTop];          // -1: none
  float w[kMaxT][kMaxTop];
  int32_t pos[kMaxE];                  // an active expert's first row of Z
  int32_t expert[kMaxE], off[kMaxE + 1];
  int32_t scan[2][kUpThreads / 32];
  int32_t active;
};

// All threads of the up kernel.  A lane holds the logits of experts lane, lane + 32, ... as
// integers in the order of their values, 0 for an expert that is off (-inf, NaN).
__device__ void route(const MoeParams& p, RouteShared& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = static_cast<int>(p.T), E = static_cast<int>(p.E), top = p.top;
  for (int i = tid; i < 2 * E; i += kUpThreads) (&sh.mask[0][0])[i] = 0;
  __syncthreads();
#pragma unroll 1
  for (int t = warp; t < T; t += kUpThreads / 32) {
    const float* row = p.logits + t * p.ldl;
    uint32_t key[kMaxE / 32];
#pragma unroll
    for (int i = 0; i < kMaxE / 32; ++i) {
      if (i * 32 >= E) {
        key[i] = 0;
        continue;
      }
      const int e = lane + 32 * i;
      const float v = e < E ? __ldg(row + e) : -INFINITY;
      const uint32_t b = __float_as_uint(v + 0.f);  // -0 and 0 are equal
      key[i] = v > -INFINITY ? ((b & 0x80000000u) ? ~b : b | 0x80000000u) : 0u;
    }
    auto value = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k); };
    float best = 0.f, sum = 0.f, chosen = 0.f, mine = 0.f;
    int my_id = -1;
#pragma unroll 1
    for (int k = 0; k < top; ++k) {
      uint32_t m = key[0];
#pragma unroll
      for (int i = 1; i < kMaxE / 32; ++i)
        if (i * 32 < E) m = max(m, key[i]);
      m = __reduce_max_sync(~0u, m);
      if (m == 0) break;
      uint32_t e = 0xFFFFFFFFu;  // the lowest expert with that logit
#pragma unroll
      for (int i = kMaxE / 32 - 1; i >= 0; --i)
        if (i * 32 < E && key[i] == m) e = lane + 32 * i;
      e = __reduce_min_sync(~0u, e);
      const float v = value(m);
      if (k == 0) {
        best = v;
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i)
          if (i * 32 < E && key[i]) sum += expf(value(key[i]) - best);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
      }
      const float w = expf(v - best);
      chosen += w;
      if (lane == k) {
        mine = w;
        my_id = static_cast<int>(e);
      }
#pragma unroll
      for (int i = 0; i < kMaxE / 32; ++i)
        if (i * 32 < E && e == static_cast<uint32_t>(lane + 32 * i)) key[i] = 0;
      if (lane == 0 && w > 0.f) atomicOr(&sh.mask[e][t >> 5], 1u << (t & 31));
    }
    if (lane < top) {
      const float by = p.renorm ? chosen : sum;
      sh.id[t][lane] = mine > 0.f ? my_id : -1;  // a weight that underflows adds nothing
      sh.w[t][lane] = mine > 0.f ? mine / by : 0.f;
    }
  }
  __syncthreads();
  // Active experts in ascending order and their rows.
  const bool mine = tid < E;
  const int count = mine ? __popc(sh.mask[tid][0]) + __popc(sh.mask[tid][1]) : 0;
  const uint32_t vote = __ballot_sync(~0u, count > 0);
  int rows = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, rows, o);
    if (lane >= o) rows += v;
  }
  if (lane == 31) {
    sh.scan[0][warp] = __popc(vote);
    sh.scan[1][warp] = rows;
  }
  __syncthreads();
  int act = __popc(vote & ((1u << lane) - 1)), first = rows - count;
#pragma unroll 1
  for (int w = 0; w < warp; ++w) {
    act += sh.scan[0][w];
    first += sh.scan[1][w];
  }
  if (count > 0) {
    sh.expert[act] = tid;
    sh.off[act] = first;
    sh.pos[tid] = first;
  }
  if (tid == kUpThreads - 1) {
    sh.active = act + (count > 0);
    sh.off[sh.active] = first + count;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ up: Z
template <int NTOK>
__global__ void __launch_bounds__(kUpThreads, 1)
    moe_up_kernel(const __grid_constant__ Maps maps, const __grid_constant__ CUtensorMap map_d, const MoeParams p) {
  using C = Cfg<NTOK>;
  constexpr int STAGES = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ RouteShared rt;
  __shared__ Pipe<STAGES> pipe;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t x_ring = ring + STAGES * W_BYTES;
  float* xch = reinterpret_cast<float*>(smem_raw + (ring - raw) + C::kRing);  // [kHalf][64]: x W_u of a tile
  volatile uint32_t* abort = &pipe.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    pipe.init();
    tma_prefetch_map(&maps.a);
    tma_prefetch_map(&maps.a2);
    tma_prefetch_map(&maps.b);
    tma_prefetch_map(&map_d);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&pipe.tmem_base), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = pipe.tmem_base;
  pdl_wait();
  route(p, rt);

  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  const uint32_t kb = static_cast<uint32_t>((p.K + BK - 1) / BK);
  const uint32_t ntiles = static_cast<uint32_t>((p.I + 63) / 64);
  const uint32_t units = static_cast<uint32_t>(rt.active) * ntiles * kb;
  const uint32_t ctas = min(units, gridDim.x);
  const bool works = blockIdx.x < ctas;
  const Split split(units, ctas > 0 ? ctas : 1);
  const uint32_t u0 = works ? split.start(blockIdx.x) : 0, u1 = works ? split.start(blockIdx.x + 1) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t u = u0; ok && u < u1;) {
        const uint32_t tile = u / kb, end = min(u1, (tile + 1) * kb);
        const int32_t e = rt.expert[tile / ntiles], n0 = static_cast<int32_t>(tile % ntiles) * 64;
        for (int32_t k = static_cast<int32_t>(u - tile * kb) * BK; u < end; ++u, k += BK) {
          const uint32_t s = it % STAGES;
          if (!mbar_wait(smem_u32(&pipe.empty[s]), ((it / STAGES) & 1u) ^ 1u, abort, p.status, kDevTimeoutProducer)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&pipe.full[s]), w = ring + s * W_BYTES;
          mbar_arrive_expect_tx(fb, W_BYTES + C::kX);
          tma_load_3d(w, &maps.a, fb, n0, k, e);
          tma_load_3d(w + W_BYTES / 2, &maps.a2, fb, n0, k, e);
          tma_load_2d(x_ring + s * C::kX, &maps.b, fb, k, 0);
          ++it;
        }
      }
      if (ok && rt.active > 0) {
        // The head of this CTA's range of the down kernel goes to L2 while this kernel ends.
        const uint32_t dkb = static_cast<uint32_t>((p.I + BK - 1) / BK), per = rt.active * dkb;
        const uint32_t dunits = static_cast<uint32_t>((p.K + 127) / 128) * per, dctas = min(dunits, gridDim.x);
        if (blockIdx.x < dctas) {
          const Split ds(dunits, dctas);
          const uint32_t d0 = ds.start(blockIdx.x), d1 = min(ds.start(blockIdx.x + 1), d0 + kPrefetch);
          for (uint32_t d = d0; d < d1; ++d) {
            const uint32_t tile = d / per, in = d - tile * per, a = in / dkb;
            const int32_t n0 = static_cast<int32_t>(tile) * 128, k = static_cast<int32_t>(in - a * dkb) * BK;
            prefetch_l2_3d(&map_d, n0, k, rt.expert[a]);
            if (n0 + 64 < p.K) prefetch_l2_3d(&map_d, n0 + 64, k, rt.expert[a]);
          }
        }
      }
      pdl_trigger();
      if (!ok) pipe.drain_loads(it, p.status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      // A = [W_g | W_u]^T tile, 64 columns each (N contiguous: MN-major), B = all tokens' X block.
      constexpr uint32_t idesc = idesc_bf16_f32(128, NTOK, true, false);
      uint32_t it = 0, lt = 0;
      bool ok = true;
      for (uint32_t u = u0; ok && u < u1; ++lt) {
        const uint32_t tile = u / kb, end = min(u1, (tile + 1) * kb), first = u;
        const uint32_t acc = lt & 1u;
        if (!mbar_wait(smem_u32(&pipe.tempty[acc]), ((lt >> 1) & 1u) ^ 1u, abort, p.status, kDevTimeoutMma)) break;
        tc_fence_after();
        for (; u < end; ++u, ++it) {
          const uint32_t s = it % STAGES;
          if (!mbar_wait(smem_u32(&pipe.full[s]), (it / STAGES) & 1u, abort, p.status, kDevTimeoutMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w0 = ring + s * W_BYTES, x0 = x_ring + s * C::kX;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_bf16(tmem_base + acc * NTOK, sdesc_sw128(w0 + k * 2048, W_BYTES / 2, 1024),
                      sdesc_sw128(x0 + k * 32, 16, 1024), idesc, (u > first || k > 0) ? 1u : 0u);
          umma_commit(smem_u32(&pipe.empty[s]));
        }
        if (ok) umma_commit(smem_u32(&pipe.tfull[acc]));
      }
      umma_commit(smem_u32(&pipe.drain));
      uint32_t never = 0;
      mbar_wait(smem_u32(&pipe.drain), 0, &never, p.status, kDevTimeoutDrain);
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, row = q * 32 + lane, etid = threadIdx.x - 64;
    const int64_t ldz = ldz_of(p.I);
    uint16_t* Z = reinterpret_cast<uint16_t*>(ws + z_at(p.T));
    float* parts = reinterpret_cast<float*>(ws + kPartsAt);
    uint32_t lt = 0;
    for (uint32_t u = u0; u < u1; ++lt) {
      const uint32_t tile = u / kb, end = min(u1, (tile + 1) * kb);
      const bool whole = end - u == kb;
      const uint32_t acc = lt & 1u;
      const int a = static_cast<int>(tile / ntiles), e = rt.expert[a];
      const int n = static_cast<int>(tile % ntiles) * 64 + (row & 63);
      const uint32_t masks[2] = {rt.mask[e][0], rt.mask[e][1]};
      // One thread waits (bounded); all 128 take the same decision after the barrier.
      if (etid == 0)
        pipe.seg_ok = mbar_wait(smem_u32(&pipe.tfull[acc]), (lt >> 1) & 1u, abort, p.status, kDevTimeoutEpilogue) ? 1u : 0u;
      epi_bar();
      if (!pipe.seg_ok) break;
      tc_fence_after();
      // z of tokens [32 h, + kHalf) of the tile from its finished sums v.
      auto finish = [&](int h, const float (&v)[C::kHalf]) {
        const uint32_t mask = masks[h];
        if (row >= 64) {
#pragma unroll
          for (int t = 0; t < C::kHalf; ++t)
            if ((mask >> t) & 1u) xch[t * 64 + row - 64] = v[t];
        }
        epi_bar();
        if (row < 64 && n < p.I) {
          const int64_t z0 = rt.off[a] + (h ? __popc(masks[0]) : 0);
#pragma unroll
          for (int t = 0; t < C::kHalf; ++t)
            if ((mask >> t) & 1u) {
              const float z = v[t] / (1.f + expf(-v[t])) * xch[t * 64 + row];
              Z[(z0 + __popc(mask & ((1u << t) - 1))) * ldz + n] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
            }
        }
        epi_bar();
      };
      // A CTA's part of a tile that began in an earlier CTA is its first, else its last.
      float* part = parts + (2 * blockIdx.x + (u0 > tile * kb ? 0 : 1)) * part_floats(p.T) + row;
#pragma unroll
      for (int h = 0; h < NTOK / C::kHalf; ++h) {
        float v[C::kHalf];
        tmem_ld<C::kHalf>(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * NTOK + h * 32, v);
        if (h == NTOK / C::kHalf - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&pipe.tempty[acc]));
        }
        if (whole) {
          finish(h, v);
        } else {
#pragma unroll
          for (int t = 0; t < C::kHalf; ++t)
            if ((masks[h] >> t) & 1u) __stcg(part + (h * 32 + t) * 128, v[t]);
        }
      }
      if (!whole) {
        // The barrier orders the CTA's stores before the ticket, whose release covers them.  A
        // CTA is the first one of at most one tile that goes on after it: its counter is the tile's.
        const uint32_t c0 = split.worker(tile * kb), c1 = split.worker((tile + 1) * kb - 1);
        epi_bar();
        if (etid == 0) {
          uint32_t* counter = reinterpret_cast<uint32_t*>(ws) + c0;
          const bool last = take_ticket(counter) == c1 - c0;
          if (last) *counter = 0;
          pipe.is_last = last;
        }
        epi_bar();
        if (pipe.is_last) {
#pragma unroll
          for (int h = 0; h < NTOK / C::kHalf; ++h) {
            float s[C::kHalf];
#pragma unroll
            for (int t = 0; t < C::kHalf; ++t) s[t] = 0.f;
            for (uint32_t c = c0; c <= c1; ++c) {
              const float* src = parts + (2 * c + (c > c0 ? 0 : 1)) * part_floats(p.T) + row;
#pragma unroll
              for (int t = 0; t < C::kHalf; ++t)
                if ((masks[h] >> t) & 1u) s[t] += __ldcg(src + (h * 32 + t) * 128);
            }
            finish(h, s);
          }
        }
        epi_bar();  // is_last is rewritten only after everyone read it
      }
      u = end;
    }
  } else if (warp == 6 && blockIdx.x == 0) {
    // ------------------------------------------------------------ the routes, for the down kernel
    Routes* out = reinterpret_cast<Routes*>(ws + kRoutesAt);
    if (lane == 0) out->active = rt.active;
    for (int i = lane; i <= rt.active; i += 32) {
      if (i < rt.active) out->expert[i] = rt.expert[i];
      out->off[i] = rt.active ? rt.off[i] : 0;
    }
    const int top = p.top, pairs = static_cast<int>(p.T) * top;
    for (int i = lane; i < pairs; i += 32) {
      const int t = i / top, e = rt.id[t][i - t * top];
      if (e < 0) continue;
      const uint32_t lo = rt.mask[e][0], hi = rt.mask[e][1], bit = (1u << (t & 31)) - 1;
      const int at = rt.pos[e] + (t < 32 ? __popc(lo & bit) : __popc(lo) + __popc(hi & bit));
      out->token[at] = t;
      out->weight[at] = rt.w[t][i - t * top];
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmem);
  }
}

// ------------------------------------------------------------------ down: Y
template <int NTOK>
__global__ void __launch_bounds__(kDownThreads, 1)
    moe_down_kernel(const __grid_constant__ Maps maps, const MoeParams p) {
  using C = Cfg<NTOK>;
  constexpr int STAGES = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Pipe<STAGES> pipe;
  __shared__ int32_t expert[kMaxE], off[kMaxE + 1], token[kMaxPairs];
  __shared__ float weight[kMaxPairs];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const uint32_t z_ring = ring + STAGES * W_BYTES;
  float* yacc = reinterpret_cast<float*>(smem_raw + (ring - raw) + C::kRing);  // [T][128]
  volatile uint32_t* abort = &pipe.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  const Routes* routes = reinterpret_cast<const Routes*>(ws + kRoutesAt);

  if (threadIdx.x == 0) {
    pipe.init();
    tma_prefetch_map(&maps.a);
    tma_prefetch_map(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&pipe.tmem_base), C::kTmem);
    tmem_relinquish();
  }
  pdl_wait();
  const int active = __ldcg(&routes->active);
  for (int i = threadIdx.x; i <= active; i += kDownThreads) {
    if (i < active) expert[i] = __ldcg(&routes->expert[i]);
    off[i] = __ldcg(&routes->off[i]);
  }
  const int rows_all = __ldcg(&routes->off[active]);
  for (int i = threadIdx.x; i < rows_all; i += kDownThreads) {
    token[i] = __ldcg(&routes->token[i]);
    weight[i] = __ldcg(&routes->weight[i]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = pipe.tmem_base;
  const int T = static_cast<int>(p.T);
  const uint32_t kb = static_cast<uint32_t>((p.I + BK - 1) / BK), per = static_cast<uint32_t>(active) * kb;
  const uint32_t units = static_cast<uint32_t>((p.K + 127) / 128) * per;
  const uint32_t ctas = min(units, gridDim.x);
  const bool works = blockIdx.x < ctas;
  const Split split(units, ctas > 0 ? ctas : 1);
  const uint32_t u0 = works ? split.start(blockIdx.x) : 0, u1 = works ? split.start(blockIdx.x + 1) : 0;

  if (active == 0) {  // no expert at all: Y = 0
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kDownThreads + threadIdx.x; i < p.T * p.K;
         i += static_cast<int64_t>(gridDim.x) * kDownThreads)
      p.Y[i / p.K * p.ldy + i % p.K] = 0;
  }
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      fence_proxy_async_global();  // Z was written by ordinary stores
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t u = u0; ok && u < u1;) {
        const uint32_t tile = u / per, in = u - tile * per, a = in / kb;
        const uint32_t end = min(u1, tile * per + (a + 1) * kb);
        const int32_t n0 = static_cast<int32_t>(tile) * 128, e = expert[a], z0 = off[a];
        const int boxes = (off[a + 1] - z0 + 15) / 16;
        for (int32_t k = static_cast<int32_t>(in - a * kb) * BK; u < end; ++u, k += BK) {
          const uint32_t s = it % STAGES;
          if (!mbar_wait(smem_u32(&pipe.empty[s]), ((it / STAGES) & 1u) ^ 1u, abort, p.status, kDevTimeoutProducer)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&pipe.full[s]), w = ring + s * W_BYTES;
          mbar_arrive_expect_tx(fb, W_BYTES + boxes * (16 * BK * 2));
          tma_load_3d(w, &maps.a, fb, n0, k, e);
          tma_load_3d(w + W_BYTES / 2, &maps.a, fb, n0 + 64, k, e);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(z_ring + s * C::kX + i * (16 * BK * 2), &maps.b, fb, k, z0 + i * 16);
          ++it;
        }
      }
      pdl_trigger();
      if (!ok) pipe.drain_loads(it, p.status);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t it = 0, lt = 0;
      bool ok = true;
      for (uint32_t u = u0; ok && u < u1; ++lt) {
        const uint32_t tile = u / per, in = u - tile * per, a = in / kb;
        const uint32_t end = min(u1, tile * per + (a + 1) * kb), first = u;
        const uint32_t boxes = (off[a + 1] - off[a] + 15) / 16;
        const uint32_t idesc = idesc_bf16_f32(128, 16 * boxes, true, false);
        const uint32_t acc = lt & 1u;
        if (!mbar_wait(smem_u32(&pipe.tempty[acc]), ((lt >> 1) & 1u) ^ 1u, abort, p.status, kDevTimeoutMma)) break;
        tc_fence_after();
        for (; u < end; ++u, ++it) {
          const uint32_t s = it % STAGES;
          if (!mbar_wait(smem_u32(&pipe.full[s]), (it / STAGES) & 1u, abort, p.status, kDevTimeoutMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w0 = ring + s * W_BYTES, z0 = z_ring + s * C::kX;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_bf16(tmem_base + acc * NTOK, sdesc_sw128(w0 + k * 2048, W_BYTES / 2, 1024),
                      sdesc_sw128(z0 + k * 32, 16, 1024), idesc, (u > first || k > 0) ? 1u : 0u);
          umma_commit(smem_u32(&pipe.empty[s]));
        }
        if (ok) umma_commit(smem_u32(&pipe.tfull[acc]));
      }
      umma_commit(smem_u32(&pipe.drain));
      uint32_t never = 0;
      mbar_wait(smem_u32(&pipe.drain), 0, &never, p.status, kDevTimeoutDrain);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, row = q * 32 + lane, etid = threadIdx.x - 64;
    float* parts = reinterpret_cast<float*>(ws + kPartsAt);
    for (int t = 0; t < T; ++t) yacc[t * 128 + row] = 0.f;  // a thread touches its column only
    uint32_t lt = 0;
    for (uint32_t u = u0; u < u1; ++lt) {
      const uint32_t tile = u / per, in = u - tile * per, a = in / kb;
      const uint32_t tile_end = (tile + 1) * per, end = min(u1, tile * per + (a + 1) * kb);
      const uint32_t acc = lt & 1u;
      const int z0 = off[a], rows = off[a + 1] - z0;
      if (etid == 0)
        pipe.seg_ok = mbar_wait(smem_u32(&pipe.tfull[acc]), (lt >> 1) & 1u, abort, p.status, kDevTimeoutEpilogue) ? 1u : 0u;
      epi_bar();
      if (!pipe.seg_ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int g = 0; g < rows; g += 16) {
        float v[16];
        tmem_ld<16>(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * NTOK + g, v);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (g + j < rows) {
            float* y = yacc + token[z0 + g + j] * 128 + row;
            *y = fmaf(weight[z0 + g + j], v[j], *y);
          }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&pipe.tempty[acc]));
      u = end;
      if (u < tile_end && u < u1) {
        epi_bar();  // seg_ok is rewritten only after everyone read it
        continue;
      }
      // ---- the column tile is done, here or as far as this CTA goes
      const int64_t n = static_cast<int64_t>(tile) * 128 + row;
      const uint32_t c0 = split.worker(tile * per), c1 = split.worker(tile_end - 1);
      bool write = true;
      if (c0 != c1) {
        float* part = parts + (2 * blockIdx.x + (u0 > tile * per ? 0 : 1)) * part_floats(p.T) + row;
        for (int t = 0; t < T; ++t) __stcg(part + t * 128, yacc[t * 128 + row]);
        epi_bar();
        if (etid == 0) {
          uint32_t* counter = reinterpret_cast<uint32_t*>(ws) + kMaxCtas + c0;
          const bool last = take_ticket(counter) == c1 - c0;
          if (last) *counter = 0;
          pipe.is_last = last;
        }
        epi_bar();
        write = pipe.is_last;
        if (write) {
          for (int t = 0; t < T; ++t) yacc[t * 128 + row] = 0.f;
          for (uint32_t c = c0; c <= c1; ++c) {
            const float* src = parts + (2 * c + (c > c0 ? 0 : 1)) * part_floats(p.T) + row;
#pragma unroll 8
            for (int t = 0; t < T; ++t) yacc[t * 128 + row] += __ldcg(src + t * 128);
          }
        }
      }
      if (write && n < p.K)
        for (int t = 0; t < T; ++t)
          p.Y[t * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(yacc[t * 128 + row]));
      for (int t = 0; t < T; ++t) yacc[t * 128 + row] = 0.f;
      epi_bar();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmem);
  }
}

template <int NTOK>
cudaError_t launch_ntok(const MoeParams& p, const Maps& up, const Maps& down, int sms, cudaStream_t s) {
  using C = Cfg<NTOK>;
  constexpr uint32_t smem_up = 1024 + C::kRing + C::kHalf * 64 * 4;
  constexpr uint32_t smem_down = 1024 + C::kRing + NTOK * 128 * 4;
  static_assert(smem_up + sizeof(RouteShared) + 512 <= 227 * 1024, "shared memory");
  static_assert(smem_down + (2 * kMaxE + 1 + 2 * kMaxPairs) * 4 + 512 <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done_up{0}, done_down{0};
  cudaError_t e = ensure_smem_attr(moe_up_kernel<NTOK>, smem_up, done_up);
  if (e != cudaSuccess) return e;
  e = ensure_smem_attr(moe_down_kernel<NTOK>, smem_down, done_down);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(sms < kMaxCtas ? sms : kMaxCtas));
  e = launch_pdl(moe_up_kernel<NTOK>, grid, dim3(kUpThreads), smem_up, s, up, down.a, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(moe_down_kernel<NTOK>, grid, dim3(kDownThreads), smem_down, s, down, p);
}

}  // namespace

int64_t moe_ws_bytes(int64_t T, int64_t I, int64_t top) {
  return z_at(T) + up256(T * top * ldz_of(I) * 2);
}

bool make_bf16_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                   uint64_t batch, uint64_t stride, uint32_t box_inner, uint32_t box_outer);

cudaError_t launch_moe(const MoeParams& p, int sms, cudaStream_t s) {
  // Experts are the third dimension; a map of one expert keeps it (its second index is never
  // loaded), so that the kernels have one form.
  const uint64_t experts = p.E > 1 ? p.E : 2;
  auto stride = [&](int64_t given, int64_t rows, int64_t ld) {
    return static_cast<uint64_t>(p.E > 1 ? given : rows * ld);
  };
  Maps up, down;
  const int ntok = ntok_of(p.T);
  const uint8_t* z = static_cast<const uint8_t*>(p.ws) + z_at(p.T);
  if (!make_bf16_map(&up.a, p.Wg, p.I, p.K, p.ldwg, experts, stride(p.strideWg, p.K, p.ldwg), 64, BK) ||
      !make_bf16_map(&up.a2, p.Wu, p.I, p.K, p.ldwu, experts, stride(p.strideWu, p.K, p.ldwu), 64, BK) ||
      !make_bf16_map(&up.b, p.X, p.K, p.T, p.ldx, 1, 0, BK, ntok) ||
      !make_bf16_map(&down.a, p.Wd, p.K, p.I, p.ldwd, experts, stride(p.strideWd, p.I, p.ldwd), 64, BK) ||
      !make_bf16_map(&down.b, z, p.I, p.T * p.top, ldz_of(p.I), 1, 0, BK, 16))
    return cudaErrorInvalidValue;
  down.a2 = down.a;
  return ntok == 16 ? launch_ntok<16>(p, up, down, sms, s)
                    : ntok == 32 ? launch_ntok<32>(p, up, down, sms, s) : launch_ntok<64>(p, up, down, sms, s);
}

}  // namespace dg
