// moe.cu -- a mixture-of-experts layer for few tokens, from the router's logits on:
//   p = softmax(logits) over the E experts; the `top` largest logits are chosen (ties: the
//   lowest expert), w = p (over the sum of the chosen p when renorm);
//   z = SiLU(x W_g[e]) * (x W_u[e]),  y = bf16(sum_e w_e (z W_d[e])).
// Products are BF16 with FP32 sums.  z enters the second product as two BF16 operands, z rounded
// and what that left over (16 significant bits together): one alone has as large an error in y
// as y's own rounding (0.0023 to 0.0027 in the mean square of y against 0.0017), and the second
// costs only a narrow product, since the weights are what is read.
//
// With at most 64 tokens every weight of a chosen expert is used a few times: reading each
// once from HBM bounds the layer.  Two kernels, one CTA per SM each, the second launched
// programmatically behind the first:
//   * up: (128 columns of W_g and of W_u, expert, 64 rows of K) units of the active experts;
//   * down: (128 columns of W_d, expert, 64 rows of I) units.  A column tile sums over experts in
//     FP32 in shared memory, one addition per expert and token.
// Both route up to 16 tokens in every CTA, a warp per token (more have a small launch of their own
// first), and cut the units evenly over the CTAs, however many experts are active.  Tiles are
// 128 columns, 256 bytes of each weight row: with 64 columns of W_g and 64 of W_u beside them
// the up kernel streamed 4.9 TB/s where this form's rows of 256 bytes reach 6.
// Units stream through a ring of TMA stages into tcgen05 with the weights as the 128-row
// operand (as they lie, N contiguous) and the tokens as the narrow one: all T tokens in the
// first product (rows of other experts are ignored: gathering them would cost more than their
// columns), an expert's own rows, 16 at a time, in the second, whose input the first writes
// sorted by expert.  The down kernel fills its ring with weights before it waits for the first.
// A tile cut between CTAs is finished by the last of them to arrive, which adds the parts in CTA
// order: results do not depend on arrival.
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
constexpr uint32_t W_BYTES = 128 * BK * 2;  // of one matrix
constexpr int kThreads = 512;        // routing: a warp per token
constexpr int kWarps = kThreads / 32;
static_assert(kMaxE == kThreads, "a thread per expert");
constexpr int kPrefetch = 16;        // units of W_d after its ring that a CTA asks L2 for early
// Small calls: a CTA is given at least this many units, as a join of many parts costs more than
// a few more units in a row (up 2, 4 or 8, us: one token, 4 of 32 experts of 1024 x 512 16.1, 15.8,
// 17.1; 6 tokens, 2 of 8 of 904 x 74 22.1, 18.2, 20.2; down 3, 4 or 8: 16.7, 15.8, 16.7 and 20.0, 18.2,
// 19.0).
constexpr uint32_t kMinUp = 4, kMinDown = 4;

// Workspace: counters (zero between calls), the tokens' choices (calls with a routing launch),
// parts of cut tiles, Z (rows sorted by expert, then the same rows' remainders).
constexpr int64_t kChoicesAt = 2048, kPartsAt = kChoicesAt + 8192;
static_assert(2 * kMaxCtas * 4 <= kChoicesAt, "counters");
constexpr int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
constexpr int ntok_of(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }
constexpr __host__ __device__ int64_t part_floats(int ntok) { return ntok * 256; }
constexpr int64_t z_at(int64_t T) { return kPartsAt + 2 * kMaxCtas * part_floats(ntok_of(T)) * 4; }
constexpr __host__ __device__ int64_t ldz_of(int64_t I) { return (I + 7) / 8 * 8; }

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

// A kernel's units, and a CTA's share of them.  CTAs work in groups of neighbours, each on its own
// one of a group's neighbouring column tiles: the rows' lines that two tiles have in common are
// then asked for by both at nearly the same time and come from HBM once.  The
// groups cut the row of (column group, expert, block of rows) units evenly; CTAs whose place in
// the last group is past the last column have a row that ends before it.
struct Share {
  uint32_t group, place, u0 = 0, u1 = 0;
  Split split;
  // `tiles` column tiles of `per` units each.
  __device__ __forceinline__ Share(uint32_t tiles, uint32_t per, uint32_t g, uint32_t least)
      : group(g), place(blockIdx.x % g), split(0, 1) {
    const uint32_t units = (tiles + g - 1) / g * per;
    const uint32_t workers = min((units + least - 1) / least, gridDim.x / g), me = blockIdx.x / g;
    if (workers == 0) return;
    split = Split(units, workers);
    if (me >= workers) return;
    const uint32_t mine = place < tiles ? ((tiles - place - 1) / g + 1) * per : 0;
    u0 = min(split.start(me), mine);
    u1 = min(split.start(me + 1), mine);
  }
  __device__ __forceinline__ uint32_t cta(uint32_t worker) const { return worker * group + place; }
  __device__ __forceinline__ uint32_t column(uint32_t t) const { return (t * group + place) * 128; }  // first, of group t
};

__device__ __forceinline__ uint32_t take_ticket(uint32_t* a) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a) : "memory");
  return old;
}
// Orders this thread's view of ordinary global stores before its TMA loads.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
// The warps that join cut tiles: all but the producer's and the MMA issuer's.
constexpr int kJoin = kThreads - 64;
__device__ __forceinline__ void join_bar() { asm volatile("bar.sync 2, %0;" ::"n"(kJoin) : "memory"); }
__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l2_3d(const CUtensorMap* map, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

struct UpMaps {
  CUtensorMap wg, wu, x;
};
struct DownMaps {
  CUtensorMap wd, z8, z16;  // Z in boxes of 8 and of 16 rows
};

template <int STAGES>
struct Pipe {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem_base, abort, is_last, seg_ok;
  uint32_t issued;  // stages that the producer filled, written when it ends
  int32_t job;  // the tile to join, -1 for none left
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
    issued = 0;
    fence_barrier_init();
  }
  // After any role gave up: the copies in flight end before the CTA does.
  __device__ void drain_loads(uint32_t* status) {
    uint32_t never = 0;
    for (uint32_t j = issued > STAGES ? issued - STAGES : 0u; j < issued; ++j)
      mbar_wait(smem_u32(&full[j % STAGES]), (j / STAGES) & 1u, &never, status, kDevTimeoutDrain);
  }
};

// One column of the accumulator: a value per lane.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, float& v) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
  v = __uint_as_float(r);
}

// ------------------------------------------------------------------ routing
struct Routes {
  uint32_t mask[kMaxE][2];             // tokens of an expert
  int16_t id[kMaxT][kMaxTop];          // -1: none
  float w[kMaxT][kMaxTop];
  int16_t pos[kMaxE];                  // an active expert's first row of Z
  int16_t expert[kMaxE], off[kMaxE + 1];  // active experts in ascending order, their first rows
  uint8_t token[kMaxPairs];            // of a row of Z
  float weight[kMaxPairs];
  int32_t scan[2][kWarps];
  int32_t active;
};

// The choices of all tokens in the workspace.
struct Choices {
  float w[kMaxT][kMaxTop];
  int16_t id[kMaxT][kMaxTop];
};
static_assert(sizeof(Choices) <= kPartsAt - kChoicesAt, "choices");

// The chosen experts of tokens warp, warp + warps, ..., a warp per token; KE * 32 >= E.  A lane holds the logits of
// experts lane, lane + 32, ... as integers in the order of their values, 0 for an expert that is
// off (-inf, NaN).  The `top`-th largest is found bit by bit from the top, by votes, stopping as
// soon as a threshold leaves exactly `top`: some 17 votes whatever `top` is.  (Taking the
// largest `top` times took 6.4 us for 48 tokens, 8 of 64 experts, by integer reductions, 8.3 us
// by shuffles.)
template <int KE, bool GLOBAL>
__device__ __forceinline__ void choose(const MoeParams& p, Routes* sh, Choices* out, int warp, int warps, int lane) {
  const int T = static_cast<int>(p.T), E = static_cast<int>(p.E), top = p.top;
  auto load = [&](int t, uint32_t (&key)[KE]) {
#pragma unroll
    for (int i = 0; i < KE; ++i) {
      const int e = lane + 32 * i;
      const float v = t < T && e < E ? __ldcg(p.logits + t * p.ldl + e) : -INFINITY;
      const uint32_t b = __float_as_uint(v + 0.f);  // -0 and 0 are equal
      key[i] = v > -INFINITY ? ((b & 0x80000000u) ? ~b : b | 0x80000000u) : 0u;
    }
  };
  auto value = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k); };
  uint32_t key[KE], next[KE];
  load(warp, next);
#pragma unroll 1
  for (int t = warp; t < T; t += warps) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < KE; ++i) {
      key[i] = next[i];
      m = max(m, key[i]);
    }
    load(t + warps, next);
    const uint32_t high = __reduce_max_sync(~0u, m), low = __reduce_min_sync(~0u, m);
    const float best = value(high);
    auto count = [&](uint32_t least) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < KE; ++i) n += __popc(__ballot_sync(~0u, key[i] >= least));
      return n;
    };
    uint32_t bar = 1;  // chosen: key > bar - 1, or some of those equal to bar
    int left = top, n = count(1);
    if (n > top) {
      // 32 numbers, which is more than `top`, reach the least of the lanes' largest: what that
      // and the largest of all begin with is known.
      uint32_t bit = high != low ? 0x80000000u >> __clz(high ^ low) : 0;
      bar = high & ~(2 * bit - (bit != 0));
      n = count(bar);
#pragma unroll 1
      for (; bit != 0 && n != top; bit >>= 1) {
        const int c = count(bar | bit);
        if (c >= top) {
          bar |= bit;
          n = c;
        }
      }
    }
    const bool tied = n > top;  // more than `top` from bar on: the lowest experts of those equal to it
    if (tied) left = top - count(bar + 1);
    float w[KE], sum = 0.f;
    int slot = 0;
#pragma unroll
    for (int i = 0; i < KE; ++i) {
      const uint32_t lower = (1u << lane) - 1;
      bool in = key[i] >= bar && key[i] > 0;
      if (tied) {
        const uint32_t equal = __ballot_sync(~0u, key[i] == bar);
        if (key[i] == bar && __popc(equal & lower) >= left) in = false;
        left -= min(left, __popc(equal));
      }
      const float x = key[i] ? expf(value(key[i]) - best) : 0.f;
      w[i] = in ? x : 0.f;
      sum += p.renorm ? w[i] : x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const float scale = 1.f / sum;  // one division in the code; the weights are within 2^-23
#pragma unroll
    for (int i = 0; i < KE; ++i) {
      const uint32_t in = __ballot_sync(~0u, w[i] > 0.f);  // a weight that underflows adds nothing
      if (w[i] > 0.f) {
        const int at = slot + __popc(in & ((1u << lane) - 1));
        (GLOBAL ? out->id : sh->id)[t][at] = static_cast<int16_t>(lane + 32 * i);
        (GLOBAL ? out->w : sh->w)[t][at] = w[i] * scale;
        if (!GLOBAL) atomicOr(&sh->mask[lane + 32 * i][t >> 5], 1u << (t & 31));
      }
      slot += __popc(in);
    }
    if (lane >= slot && lane < top) (GLOBAL ? out->id : sh->id)[t][lane] = -1;
  }
}

template <bool GLOBAL>
__device__ __forceinline__ void choose_all(const MoeParams& p, Routes* sh, Choices* out, int warp, int warps, int lane) {
  if (p.E <= 64) choose<2, GLOBAL>(p, sh, out, warp, warps, lane);
  else if (p.E <= 128) choose<4, GLOBAL>(p, sh, out, warp, warps, lane);
  else choose<16, GLOBAL>(p, sh, out, warp, warps, lane);
}

// More than 16 tokens: a launch of its own, a warp per token.  In every CTA of the other two
// kernels the same took 7 us for 48 or 64 tokens of 64 experts, twice; for up to 16 tokens (one a
// warp) it takes 2 to 3 us there, which this launch would not beat.
constexpr int kRouteWarps = 4;
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_kernel(const MoeParams p) {
  pdl_wait();
  pdl_trigger();
  Choices* out = reinterpret_cast<Choices*>(static_cast<uint8_t*>(p.ws) + kChoicesAt);
  choose_all<true>(p, nullptr, out, blockIdx.x * kRouteWarps + (threadIdx.x >> 5), gridDim.x * kRouteWarps, threadIdx.x & 31);
}

// All threads; the masks are zero and that is visible.  Logits and choices are read from L2: the
// down kernel routes before the up kernel has ended, and they were complete before that one
// started anything.
template <int NTOK>
__device__ __forceinline__ void route(const MoeParams& p, Routes& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = static_cast<int>(p.E), top = p.top;
  if constexpr (NTOK == 16) {
    choose_all<false>(p, &sh, nullptr, warp, kWarps, lane);
  } else {
    const Choices* in = reinterpret_cast<const Choices*>(static_cast<const uint8_t*>(p.ws) + kChoicesAt);
    for (int i = tid; i < static_cast<int>(p.T) * kMaxTop; i += kThreads) {
      const int t = i / kMaxTop, k = i % kMaxTop;
      if (k >= top) continue;
      const int16_t e = __ldcg(&in->id[t][k]);
      sh.id[t][k] = e;
      sh.w[t][k] = __ldcg(&in->w[t][k]);
      if (e >= 0) atomicOr(&sh.mask[e][t >> 5], 1u << (t & 31));
    }
  }
  __syncthreads();
  // Active experts in ascending order and their rows: a thread per expert.
  const int count = tid < E ? __popc(sh.mask[tid][0]) + __popc(sh.mask[tid][1]) : 0;
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
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {  // (to its own warp only, one load waits for another: 0.7 us)
    act += w < warp ? sh.scan[0][w] : 0;
    first += w < warp ? sh.scan[1][w] : 0;
  }
  if (count > 0) {
    sh.expert[act] = static_cast<int16_t>(tid);
    sh.off[act] = sh.pos[tid] = static_cast<int16_t>(first);
  }
  if (tid == kThreads - 1) {
    sh.active = act + (count > 0);
    sh.off[sh.active] = static_cast<int16_t>(first + count);
  }
  __syncthreads();
  const int pairs = static_cast<int>(p.T) * top;
#pragma unroll 1
  for (int i = tid; i < pairs; i += kThreads) {
    const int t = i / top, e = sh.id[t][i - t * top];
    if (e < 0) continue;
    const uint32_t lo = sh.mask[e][0], bit = (1u << (t & 31)) - 1;
    const int at = sh.pos[e] + (t < 32 ? __popc(lo & bit) : __popc(lo) + __popc(sh.mask[e][1] & bit));
    sh.token[at] = static_cast<uint8_t>(t);
    sh.weight[at] = sh.w[t][i - t * top];
  }
  __syncthreads();
}

// ------------------------------------------------------------------ up: Z
template <int NTOK>
struct UpCfg {
  static constexpr int kStages = NTOK == 16 ? 6 : 5;
  static constexpr uint32_t kX = NTOK * BK * 2;
  static constexpr uint32_t kStage = 2 * W_BYTES + kX;
  static constexpr uint32_t kTmem = 4 * NTOK;  // (gate, up) twice
  static constexpr uint32_t kSmem = 1024 + kStages * kStage;
  static_assert(kSmem + sizeof(Routes) + 512 <= 227 * 1024, "shared memory");
};

template <int NTOK>
__global__ void __launch_bounds__(kThreads, 1) moe_up_kernel(const __grid_constant__ UpMaps maps, const MoeParams p) {
  using C = UpCfg<NTOK>;
  constexpr int STAGES = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Routes rt;
  __shared__ Pipe<STAGES> pipe;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  volatile uint32_t* abort = &pipe.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  rt.mask[threadIdx.x][0] = rt.mask[threadIdx.x][1] = 0;  // kMaxE == kThreads
  if (threadIdx.x == 0) {
    pipe.init();
    tma_prefetch_map(&maps.wg);
    tma_prefetch_map(&maps.wu);
    tma_prefetch_map(&maps.x);
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
  // The down kernel's CTAs take an SM each as this kernel's leave it, route, and fill their rings.
  pdl_trigger();
  route<NTOK>(p, rt);

  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  const uint32_t kb = static_cast<uint32_t>((p.K + BK - 1) / BK), active = static_cast<uint32_t>(rt.active);
  const Share share(static_cast<uint32_t>((p.I + 127) / 128), active * kb, p.up_group, kMinUp);
  const uint32_t u0 = share.u0, u1 = share.u1;

  const int64_t ldz = ldz_of(p.I);
  uint16_t* Z = reinterpret_cast<uint16_t*>(ws + (kPartsAt + 2 * kMaxCtas * part_floats(NTOK) * 4));
  const int64_t rest = p.T * p.top * ldz;  // from z rounded to its remainder
  auto put_z = [&](int row, int64_t n, float g, float up) {
    const float z = g / (1.f + expf(-g)) * up;
    const __nv_bfloat16 hi = __float2bfloat16_rn(z);
    const float left = z - __bfloat162float(hi);
    // What passes BF16's range is Inf, and has no remainder (Inf - Inf would make a NaN of its sums).
    const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(left) < INFINITY ? left : 0.f);
    Z[row * ldz + n] = __bfloat16_as_ushort(hi);
    Z[rest + row * ldz + n] = __bfloat16_as_ushort(lo);
  };
  // Adds a tile's parts in CTA order, four columns of one row a thread, and writes their Z.
  auto join = [&](uint32_t tile) {
    const uint32_t c0 = share.split.worker(tile * kb), c1 = share.split.worker((tile + 1) * kb - 1);
    const int a = static_cast<int>(tile % active), z0 = rt.off[a], rows = rt.off[a + 1] - z0;
    const float* parts = reinterpret_cast<const float*>(ws + kPartsAt);
#pragma unroll 1
    for (int i = threadIdx.x - 64; i < rows * 32; i += kJoin) {
      const int r = i >> 5, c4 = (i & 31) * 4;
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
#pragma unroll 1
      for (uint32_t c = c0; c <= c1; c += 4) {
        float4 v[4], w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float* src = parts + (2 * share.cta(c + x) + (c + x > c0 ? 0 : 1)) * part_floats(NTOK) + r * 256 + c4;
          const bool in = c + x <= c1;
          v[x] = in ? __ldcg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
          w[x] = in ? __ldcg(reinterpret_cast<const float4*>(src + 128)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          g.x += v[x].x; g.y += v[x].y; g.z += v[x].z; g.w += v[x].w;
          u.x += w[x].x; u.y += w[x].y; u.z += w[x].z; u.w += w[x].w;
        }
      }
      const float gs[4] = {g.x, g.y, g.z, g.w}, us[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = static_cast<int64_t>(share.column(tile / active)) + c4 + j;
        if (n < p.I) put_z(z0 + r, n, gs[j], us[j]);
      }
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t u = u0; ok && u < u1;) {
        const uint32_t tile = u / kb, end = min(u1, (tile + 1) * kb);
        const int32_t e = rt.expert[tile % active], n0 = static_cast<int32_t>(share.column(tile / active));
        for (int32_t k = static_cast<int32_t>(u - tile * kb) * BK; u < end; ++u, k += BK) {
          const uint32_t s = it % STAGES;
          if (!mbar_wait(smem_u32(&pipe.empty[s]), ((it / STAGES) & 1u) ^ 1u, abort, p.status, kDevTimeoutProducer)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&pipe.full[s]), w = ring + s * C::kStage;
          mbar_arrive_expect_tx(fb, C::kStage);
          tma_load_3d(w, &maps.wg, fb, n0, k, e);
          tma_load_3d(w + W_BYTES / 2, &maps.wg, fb, n0 + 64, k, e);
          tma_load_3d(w + W_BYTES, &maps.wu, fb, n0, k, e);
          tma_load_3d(w + W_BYTES * 3 / 2, &maps.wu, fb, n0 + 64, k, e);
          tma_load_2d(w + 2 * W_BYTES, &maps.x, fb, k, 0);
          ++it;
        }
      }
      pipe.issued = it;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      // A = W_g^T, W_u^T tiles (N contiguous: MN-major), B = all tokens' X block.
      constexpr uint32_t idesc = idesc_bf16_f32(128, NTOK, true, false);
      uint32_t it = 0, lt = 0;
      bool ok = true;
      for (uint32_t u = u0; ok && u < u1; ++lt) {
        const uint32_t tile = u / kb, end = min(u1, (tile + 1) * kb), first = u;
        const uint32_t acc = lt & 1u;
        if (!mbar_wait(smem_u32(&pipe.tempty[acc]), ((lt >> 1) & 1u) ^ 1u, abort, p.status, kDevTimeoutMma)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * 2 * NTOK;
        for (; u < end; ++u, ++it) {
          const uint32_t s = it % STAGES;
          if (!mbar_wait(smem_u32(&pipe.full[s]), (it / STAGES) & 1u, abort, p.status, kDevTimeoutMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w0 = ring + s * C::kStage, x0 = w0 + 2 * W_BYTES;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k) {
            const uint64_t bdesc = sdesc_sw128(x0 + k * 32, 16, 1024);
            const uint32_t add = (u > first || k > 0) ? 1u : 0u;
            umma_bf16(d, sdesc_sw128(w0 + k * 2048, W_BYTES / 2, 1024), bdesc, idesc, add);
            umma_bf16(d + NTOK, sdesc_sw128(w0 + W_BYTES + k * 2048, W_BYTES / 2, 1024), bdesc, idesc, add);
          }
          if (p.fault != 1) umma_commit(smem_u32(&pipe.empty[s]));
        }
        if (ok) umma_commit(smem_u32(&pipe.tfull[acc]));
      }
      umma_commit(smem_u32(&pipe.drain));
      uint32_t never = 0;
      mbar_wait(smem_u32(&pipe.drain), 0, &never, p.status, kDevTimeoutDrain);
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue: a thread per column
    const int q = warp & 3, row = q * 32 + lane, etid = threadIdx.x - 64;
    float* parts = reinterpret_cast<float*>(ws + kPartsAt) + row;
    uint32_t lt = 0;
    for (uint32_t u = u0; u < u1; ++lt) {
      const uint32_t tile = u / kb, end = min(u1, (tile + 1) * kb);
      const bool whole = end - u == kb;
      const uint32_t acc = lt & 1u;
      const int a = static_cast<int>(tile % active), z0 = rt.off[a], rows = rt.off[a + 1] - z0;
      const int64_t n = static_cast<int64_t>(share.column(tile / active)) + row;
      // One thread waits (bounded); all 128 take the same decision after the barrier.
      if (etid == 0)
        pipe.seg_ok = mbar_wait(smem_u32(&pipe.tfull[acc]), (lt >> 1) & 1u, abort, p.status, kDevTimeoutEpilogue) ? 1u : 0u;
      epi_bar();
      if (!pipe.seg_ok) break;
      tc_fence_after();
      auto store = [&](int r, float g, float up) {
        if (n < p.I) put_z(z0 + r, n, g, up);
      };
      // A CTA's part of a tile that began in an earlier CTA is its first, else its last.
      float* part = parts + (2 * blockIdx.x + (u0 > tile * kb ? 0 : 1)) * part_floats(NTOK);
      const uint32_t t0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 2 * NTOK;
      constexpr int B = 8;  // rows at a time
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += B) {
        float g[B], up[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
          const uint32_t t = rt.token[min(z0 + r0 + j, kMaxPairs - 1)] & (NTOK - 1);  // past the rows: any
          tmem_ld1(t0 + t, g[j]);
          tmem_ld1(t0 + NTOK + t, up[j]);
        }
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < B; ++j) {
          if (r0 + j >= rows) break;
          if (whole) {
            store(r0 + j, g[j], up[j]);
          } else {
            __stcg(part + (r0 + j) * 256, g[j]);
            __stcg(part + (r0 + j) * 256 + 128, up[j]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&pipe.tempty[acc]));
      if (!whole) {
        // The barrier orders the CTA's stores before the ticket, whose release covers them.  A
        // CTA is the first one of at most one tile that goes on after it: its counter is the tile's.
        const uint32_t c0 = share.split.worker(tile * kb), c1 = share.split.worker((tile + 1) * kb - 1);
        epi_bar();
        if (etid == 0) {
          uint32_t* counter = reinterpret_cast<uint32_t*>(ws) + share.cta(c0);
          const bool last = take_ticket(counter) == c1 - c0;
          if (last) *counter = 0;
          pipe.is_last = last;
        }
        epi_bar();
        if (pipe.is_last) {
          if (etid == 0) pipe.job = static_cast<int32_t>(tile);
          join_bar();  // the other warps take the job
          join(tile);
          join_bar();
        }
      }
      epi_bar();  // seg_ok and is_last are rewritten only after everyone read them
      u = end;
    }
    if (etid == 0) pipe.job = -1;
    join_bar();
  } else {
    for (;;) {
      join_bar();
      const int32_t tile = pipe.job;
      if (tile < 0) break;
      join(static_cast<uint32_t>(tile));
      join_bar();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && pipe.abort) pipe.drain_loads(p.status);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmem);
  }
}

// ------------------------------------------------------------------ down: Y
template <int NTOK>
struct DownCfg {
  static constexpr int kStages = NTOK == 64 ? 5 : NTOK == 32 ? 7 : 8;
  static constexpr uint32_t kZ = NTOK * BK * 2;
  static constexpr uint32_t kStage = W_BYTES + 2 * kZ;
  static constexpr uint32_t kTmem = 4 * NTOK;  // (z, its remainders) twice
  static constexpr uint32_t kSmem = 1024 + kStages * kStage + NTOK * 128 * 4;
  static_assert(kSmem + sizeof(Routes) + 512 <= 227 * 1024, "shared memory");
};

// The narrow operand of an expert with `rows` tokens is its rows of z, then as many rows of
// their remainders: up to 8 tokens share one 16-row operand.
__device__ __forceinline__ int padded(int rows) { return rows <= 8 ? 8 : (rows + 15) / 16 * 16; }

template <int NTOK>
__global__ void __launch_bounds__(kThreads, 1) moe_down_kernel(const __grid_constant__ DownMaps maps, const MoeParams p) {
  using C = DownCfg<NTOK>;
  constexpr int STAGES = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Routes rt;
  __shared__ Pipe<STAGES> pipe;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  float* yacc = reinterpret_cast<float*>(smem_raw + (ring - raw) + STAGES * C::kStage);  // [T][128]
  volatile uint32_t* abort = &pipe.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  rt.mask[threadIdx.x][0] = rt.mask[threadIdx.x][1] = 0;  // kMaxE == kThreads
  if (threadIdx.x == 0) {
    pipe.init();
    tma_prefetch_map(&maps.wd);
    tma_prefetch_map(&maps.z8);
    tma_prefetch_map(&maps.z16);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&pipe.tmem_base), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = pipe.tmem_base;
  route<NTOK>(p, rt);  // before the wait for the up kernel: see there
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  const int T = static_cast<int>(p.T), active = rt.active;
  const uint32_t kb = static_cast<uint32_t>((p.I + BK - 1) / BK), per = static_cast<uint32_t>(active) * kb;
  const Share share(static_cast<uint32_t>((p.K + 127) / 128), per, p.down_group, kMinDown);
  const uint32_t u0 = share.u0, u1 = share.u1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      // A place in the row of units; stepping needs no division (with two a unit this thread,
      // not HBM, set the pace where L2 already had the weights).
      struct Place {
        int32_t n0, k, a;
      };
      const int32_t k_end = static_cast<int32_t>(kb) * BK;
      auto step = [&](Place& x) {
        x.k += BK;
        if (x.k < k_end) return;
        x.k = 0;
        if (++x.a == active) {
          x.a = 0;
          x.n0 += 128 * static_cast<int32_t>(p.down_group);
        }
      };
      constexpr uint32_t kRow = BK * 2;  // bytes of a row of Z in a stage
      auto load_w = [&](uint32_t s, const Place& x) {
        const uint32_t fb = smem_u32(&pipe.full[s]), w = ring + s * C::kStage;
        mbar_arrive_expect_tx(fb, W_BYTES + 2 * padded(rt.off[x.a + 1] - rt.off[x.a]) * kRow);
        tma_load_3d(w, &maps.wd, fb, x.n0, x.k, rt.expert[x.a]);
        tma_load_3d(w + W_BYTES / 2, &maps.wd, fb, x.n0 + 64, x.k, rt.expert[x.a]);
      };
      auto load_z = [&](uint32_t s, const Place& x) {
        const uint32_t fb = smem_u32(&pipe.full[s]), z = ring + s * C::kStage + W_BYTES;
        const int32_t row = rt.off[x.a], rest = static_cast<int32_t>(p.T) * p.top, half = padded(rt.off[x.a + 1] - row);
        if (half == 8) {
          tma_load_2d(z, &maps.z8, fb, x.k, row);
          tma_load_2d(z + 8 * kRow, &maps.z8, fb, x.k, rest + row);
          return;
        }
        for (int i = 0; i < half; i += 16) {
          tma_load_2d(z + i * kRow, &maps.z16, fb, x.k, row + i);
          tma_load_2d(z + (half + i) * kRow, &maps.z16, fb, x.k, rest + row + i);
        }
      };
      const uint32_t tile0 = per ? u0 / per : 0, a0 = per ? (u0 - tile0 * per) / kb : 0;
      const Place first = {static_cast<int32_t>(share.column(tile0)), static_cast<int32_t>(u0 - tile0 * per - a0 * kb) * BK,
                           static_cast<int32_t>(a0)};
      // The ring's first weights come while the up kernel ends; its Z after the wait.
      const uint32_t ahead = min(u1 - u0, static_cast<uint32_t>(STAGES));
      Place w = first;
      for (uint32_t i = 0; i < ahead; ++i, step(w)) load_w(i, w);
      // And L2 is asked for what follows: HBM streams on while the last up CTAs end.
      const uint32_t asked = min(u1 - u0 - ahead, static_cast<uint32_t>(kPrefetch));
      Place l2 = w;
      for (uint32_t i = 0; i < asked; ++i, step(l2)) {
        prefetch_l2_3d(&maps.wd, l2.n0, l2.k, rt.expert[l2.a]);
        if (l2.n0 + 64 < p.K) prefetch_l2_3d(&maps.wd, l2.n0 + 64, l2.k, rt.expert[l2.a]);
      }
      pdl_wait();
      fence_proxy_async_global();  // Z was written by ordinary stores
      Place z = first;
      for (uint32_t i = 0; i < ahead; ++i, step(z)) load_z(i, z);
      uint32_t it = ahead;
      for (uint32_t u = u0 + ahead; u < u1; ++u, ++it, step(w)) {
        const uint32_t s = it % STAGES;
        if (!mbar_wait(smem_u32(&pipe.empty[s]), ((it / STAGES) & 1u) ^ 1u, abort, p.status, kDevTimeoutProducer)) break;
        load_w(s, w);
        load_z(s, w);
      }
      pdl_trigger();
      pipe.issued = it;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      pdl_wait();  // so that its bounded waits start when the data can come
      uint32_t it = 0, lt = 0;
      bool ok = true;
      for (uint32_t u = u0; ok && u < u1; ++lt) {
        const uint32_t tile = u / per, in = u - tile * per, a = in / kb;
        const uint32_t end = min(u1, tile * per + (a + 1) * kb), first = u;
        const uint32_t idesc = idesc_bf16_f32(128, 2 * padded(rt.off[a + 1] - rt.off[a]), true, false);
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
          const uint32_t w0 = ring + s * C::kStage, z0 = w0 + W_BYTES;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            umma_bf16(tmem_base + acc * 2 * NTOK, sdesc_sw128(w0 + k * 2048, W_BYTES / 2, 1024),
                      sdesc_sw128(z0 + k * 32, 16, 1024), idesc, (u > first || k > 0) ? 1u : 0u);
          if (p.fault != 1) umma_commit(smem_u32(&pipe.empty[s]));
        }
        if (ok) umma_commit(smem_u32(&pipe.tfull[acc]));
      }
      umma_commit(smem_u32(&pipe.drain));
      uint32_t never = 0;
      mbar_wait(smem_u32(&pipe.drain), 0, &never, p.status, kDevTimeoutDrain);
    }
  } else {
    pdl_wait();
    float* parts = reinterpret_cast<float*>(ws + kPartsAt);
    const int jtid = threadIdx.x - 64;  // of those that join tiles
    if (active == 0)  // no expert at all: Y = 0
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * kJoin + jtid; i < p.T * p.K; i += static_cast<int64_t>(gridDim.x) * kJoin)
        p.Y[i / p.K * p.ldy + i % p.K] = 0;
    // Adds a tile's parts in CTA order, four columns of one token a thread, and writes them.
    auto join = [&](uint32_t tile) {
      const uint32_t c0 = share.split.worker(tile * per), c1 = share.split.worker((tile + 1) * per - 1);
#pragma unroll 1
      for (int i = jtid; i < T * 32; i += kJoin) {
        const int t = i >> 5, c4 = (i & 31) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (uint32_t c = c0; c <= c1; c += 12) {
          float4 v[12];
#pragma unroll
          for (int x = 0; x < 12; ++x)
            v[x] = c + x <= c1 ? __ldcg(reinterpret_cast<const float4*>(
                                     parts + (2 * share.cta(c + x) + (c + x > c0 ? 0 : 1)) * part_floats(NTOK) + t * 128 + c4))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < 12; ++x) {
            s.x += v[x].x;
            s.y += v[x].y;
            s.z += v[x].z;
            s.w += v[x].w;
          }
        }
        const float y[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = static_cast<int64_t>(share.column(tile)) + c4 + j;
          if (n < p.K) p.Y[t * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(y[j]));
        }
      }
    };
    if (warp < 6) {
      // ---------------------------------------------------------- epilogue: a thread per column
      const int q = warp & 3, row = q * 32 + lane, etid = threadIdx.x - 64;
      for (int t = 0; t < T; ++t) yacc[t * 128 + row] = 0.f;  // a thread touches its column only
      uint32_t lt = 0;
      for (uint32_t u = u0; u < u1; ++lt) {
        const uint32_t tile = u / per, in = u - tile * per, a = in / kb;
        const uint32_t tile_end = (tile + 1) * per, end = min(u1, tile * per + (a + 1) * kb);
        const uint32_t acc = lt & 1u;
        const int z0 = rt.off[a], rows = rt.off[a + 1] - z0;
        if (etid == 0)
          pipe.seg_ok = mbar_wait(smem_u32(&pipe.tfull[acc]), (lt >> 1) & 1u, abort, p.status, kDevTimeoutEpilogue) ? 1u : 0u;
        epi_bar();
        if (!pipe.seg_ok) break;
        tc_fence_after();
        const int half = padded(rows);
        const uint32_t t0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 2 * NTOK;
        auto add = [&](int r, uint32_t z, uint32_t rest) {
          float* y = yacc + rt.token[z0 + r] * 128 + row;
          *y = fmaf(rt.weight[z0 + r], __uint_as_float(z) + __uint_as_float(rest), *y);
        };
        if (half == 8) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(t0, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < rows) add(j, v[j], v[8 + j]);
        } else {
#pragma unroll 1
          for (int g = 0; g < rows; g += 16) {
            uint32_t v[16], w[16];
            tmem_ld_32x32b_x16(t0 + g, v);
            tmem_ld_32x32b_x16(t0 + half + g, w);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (g + j < rows) add(g + j, v[j], w[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&pipe.tempty[acc]));
        u = end;
        if (u == tile_end || u == u1) {
          // ---- the column tile is done, here or as far as this CTA goes
          const int64_t n = static_cast<int64_t>(share.column(tile)) + row;
          const uint32_t c0 = share.split.worker(tile * per), c1 = share.split.worker(tile_end - 1);
          if (c0 == c1) {
            for (int t = 0; t < T; ++t) {
              if (n < p.K) p.Y[t * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(yacc[t * 128 + row]));
              yacc[t * 128 + row] = 0.f;
            }
          } else {
            float* part = parts + (2 * blockIdx.x + (u0 > tile * per ? 0 : 1)) * part_floats(NTOK) + row;
            for (int t = 0; t < T; ++t) {
              __stcg(part + t * 128, yacc[t * 128 + row]);
              yacc[t * 128 + row] = 0.f;
            }
            // Barrier, ticket and counter as in the up kernel.
            epi_bar();
            if (etid == 0) {
              uint32_t* counter = reinterpret_cast<uint32_t*>(ws) + kMaxCtas + share.cta(c0);
              const bool last = take_ticket(counter) == c1 - c0;
              if (last) *counter = 0;
              pipe.is_last = last;
              if (last) pipe.job = static_cast<int32_t>(tile);
            }
            epi_bar();
            if (pipe.is_last) {
              join_bar();  // the other warps take the job
              join(tile);
              join_bar();
            }
          }
        }
        epi_bar();  // seg_ok and is_last are rewritten only after everyone read them
      }
      if (etid == 0) pipe.job = -1;
      join_bar();
    } else {
      for (;;) {
        join_bar();
        const int32_t tile = pipe.job;
        if (tile < 0) break;
        join(static_cast<uint32_t>(tile));
        join_bar();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && pipe.abort) pipe.drain_loads(p.status);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmem);
  }
}

template <int NTOK>
cudaError_t launch_ntok(const MoeParams& p, const UpMaps& up, const DownMaps& down, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> done_up{0}, done_down{0};
  cudaError_t e = ensure_smem_attr(moe_up_kernel<NTOK>, UpCfg<NTOK>::kSmem, done_up);
  if (e != cudaSuccess) return e;
  e = ensure_smem_attr(moe_down_kernel<NTOK>, DownCfg<NTOK>::kSmem, done_down);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(sms < kMaxCtas ? sms : kMaxCtas)), block(kThreads);
  if (NTOK > 16) {
    const unsigned ctas = static_cast<unsigned>((p.T + kRouteWarps - 1) / kRouteWarps);
    e = launch_pdl(moe_route_kernel, dim3(ctas), dim3(32 * kRouteWarps), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(moe_up_kernel<NTOK>, grid, block, UpCfg<NTOK>::kSmem, s, up, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(moe_down_kernel<NTOK>, grid, block, DownCfg<NTOK>::kSmem, s, down, p);
}

}  // namespace

int64_t moe_ws_bytes(int64_t T, int64_t I, int64_t top) {
  return z_at(T) + up256(2 * T * top * ldz_of(I) * 2);
}

bool make_bf16_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                   uint64_t batch, uint64_t stride, uint32_t box_inner, uint32_t box_outer);

// CTAs of a group: one where rows start on the 128-byte lines that HBM is read in, so that column
// tiles share none; otherwise 8, or what a row has tiles for (48 tokens, 61 active experts of
// 2048 x 1000, 1160 and 700, us: single CTAs 152, 191, 113, pairs 149, 177, 109, fours 145, 179,
// 108, eights 144, 174, 108; 718 MB came from HBM for the first one's 500 MB of W_g and W_u when
// neighbouring tiles were read far apart in time, which took 172).
uint32_t group_of(int64_t cols, int sms, bool lines) {
  const int64_t tiles = (cols + 127) / 128;
  uint32_t g = lines ? 1 : 8;
  while (g > tiles || g > static_cast<uint32_t>(sms)) g /= 2;
  return g > 0 ? g : 1;
}

cudaError_t launch_moe(const MoeParams& call, int sms, cudaStream_t s) {
  MoeParams p = call;
  p.fault = g_fault_injection;
  auto aligned = [&](const uint16_t* w, int64_t ld, int64_t stride, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(w) % bytes == 0 && ld * 2 % bytes == 0 && (p.E == 1 || stride * 2 % bytes == 0);
  };
  p.up_group = group_of(p.I, sms, aligned(p.Wg, p.ldwg, p.strideWg, 128) && aligned(p.Wu, p.ldwu, p.strideWu, 128));
  p.down_group = group_of(p.K, sms, aligned(p.Wd, p.ldwd, p.strideWd, 128));
  // Experts are the third dimension; a map of one expert keeps it (its second index is never
  // loaded), so that the kernels have one form.
  const uint64_t experts = p.E > 1 ? p.E : 2;
  auto weights = [&](CUtensorMap* map, const uint16_t* w, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
    const bool lines = aligned(w, ld, stride, 256);
    if (p.E == 1) stride = rows * ld;
    // Rows that start on 256-byte lines are read in whole ones.  Otherwise L2 is to fetch the
    // sectors asked for only: with 256-byte fetches the two ends of every row's 256 bytes bring
    // lines of which little is used before they are gone (rows of 2000 bytes: 868 MB read for 500).
    return make_tile_map_l2(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, w, cols, rows, ld, experts, stride, 64, BK,
                         CU_TENSOR_MAP_SWIZZLE_128B, 1,
                         lines ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE);
  };
  UpMaps up;
  DownMaps down;
  const int ntok = ntok_of(p.T);
  const uint8_t* z = static_cast<const uint8_t*>(p.ws) + z_at(p.T);
  if (!weights(&up.wg, p.Wg, p.K, p.I, p.ldwg, p.strideWg) || !weights(&up.wu, p.Wu, p.K, p.I, p.ldwu, p.strideWu) ||
      !weights(&down.wd, p.Wd, p.I, p.K, p.ldwd, p.strideWd) ||
      !make_bf16_map(&up.x, p.X, p.K, p.T, p.ldx, 1, 0, BK, ntok) ||
      !make_bf16_map(&down.z8, z, p.I, 2 * p.T * p.top, ldz_of(p.I), 1, 0, BK, 8) ||
      !make_bf16_map(&down.z16, z, p.I, 2 * p.T * p.top, ldz_of(p.I), 1, 0, BK, 16))
    return cudaErrorInvalidValue;
  return ntok == 16 ? launch_ntok<16>(p, up, down, sms, s)
                    : ntok == 32 ? launch_ntok<32>(p, up, down, sms, s) : launch_ntok<64>(p, up, down, sms, s);
}

}  // namespace dg
