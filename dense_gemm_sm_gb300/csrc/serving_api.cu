// serving_api.cu -- the C ABI of the serving operators: argument checks and launches.  Every
// check that needs no GPU comes before the first CUDA call, so a refused call enqueues nothing
// and touches no device.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "serving.h"

namespace dg {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

dg_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DG_OK : DG_ERR_CUDA; }

bool is_type(dg_out t) { return t == DG_OUT_BF16 || t == DG_OUT_F32; }

dg_status check_norm(int64_t rows, int64_t cols, const void* X, int64_t ldx, dg_out x_type, const void* R,
                     int64_t ldr, dg_out r_type, const void* H, int64_t ldh, const uint16_t* gain, float eps,
                     const void* Y, int64_t ldy) {
  if (rows < 0 || cols < 0 || !is_type(x_type) || !is_type(r_type)) return DG_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return DG_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return DG_OK;
  if (ldx < cols || ldy < cols || !X || !gain || !Y) return DG_ERR_INVALID_ARG;
  if ((R == nullptr) != (H == nullptr)) return DG_ERR_INVALID_ARG;
  if (R && (ldr < cols || ldh < cols)) return DG_ERR_INVALID_ARG;
  if (rows > INT32_MAX || cols > INT32_MAX) return DG_ERR_UNSUPPORTED;
  if (!aligned(X, x_type == DG_OUT_F32 ? 4 : 2) || !aligned(gain, 2)) return DG_ERR_MISALIGNED;
  const uintptr_t rb = r_type == DG_OUT_F32 ? 4 : 2;
  if (R && (!aligned(R, rb) || !aligned(H, rb))) return DG_ERR_MISALIGNED;
  return DG_OK;
}

dg_status run_norm(int64_t rows, int64_t cols, const void* X, int64_t ldx, dg_out x_type, const void* R,
                   int64_t ldr, dg_out r_type, void* H, int64_t ldh, const uint16_t* gain, float eps, void* Y,
                   int64_t ldy, float* scales, void* stream) {
  NormParams p;
  p.rows = rows; p.cols = cols;
  p.X = X; p.ldx = ldx;
  p.R = R; p.ldr = ldr;
  p.H = H; p.ldh = ldh;
  p.gain = gain; p.eps = eps;
  p.Y = Y; p.ldy = ldy;
  p.scales = scales;
  // Eight elements a step: 16-byte rows of BF16, two 16-byte words of FP32, 8 bytes of codes.
  const bool vec = aligned(X, 16) && ldx % 8 == 0 && aligned(gain, 16) &&
                   (!R || (aligned(R, 16) && aligned(H, 16) && ldr % 8 == 0 && ldh % 8 == 0)) &&
                   aligned(Y, scales ? 8 : 16) && ldy % 8 == 0;
  return from_cuda(launch_rmsnorm(p, x_type == DG_OUT_F32, r_type == DG_OUT_F32, vec, static_cast<cudaStream_t>(stream)));
}

// Sizes are held against their limits before anything is multiplied with them.
constexpr int32_t kMaxPage = 4096, kMaxCacheHeads = 4096;
constexpr int64_t kMaxAttn = 65536;  // sequences, queries of one, query heads

bool attention_takes(int64_t batch, int64_t Lq, int64_t heads_q) {
  return batch <= kMaxAttn && Lq <= kMaxAttn && heads_q <= kMaxAttn && batch * Lq * heads_q <= INT32_MAX;
}

// n > 0 rows of `width` elements, ld apart, within `span` elements (no product can overflow).
bool rows_fit(int64_t n, int64_t ld, int64_t width, int64_t span) {
  return span >= width && (n == 1 || ld <= (span - width) / (n - 1));
}

bool moe_takes(int64_t T, int64_t K, int64_t I, int64_t E, int64_t top) {
  if (T > 64 || top > 16 || E > 512 || K > INT32_MAX || I > INT32_MAX) return false;
  // Units of 64 x 128 weights of all experts are counted in 31 bits.
  const int64_t kb = (K + 63) / 64, ib = (I + 63) / 64;
  return kb <= INT32_MAX / ib / E;
}

// The cache itself: DG_OK when its pages can be addressed.
dg_status check_cache(const dg_kv4_cache* c) {
  if (!c || c->pages < 0 || c->page_size <= 0 || c->heads <= 0 || c->d <= 0) return DG_ERR_INVALID_ARG;
  if (c->page_size % kKv4Tokens != 0) return DG_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return DG_ERR_UNSUPPORTED;
  if (c->page_size > kMaxPage || c->heads > kMaxCacheHeads || c->pages > INT32_MAX) return DG_ERR_UNSUPPORTED;
  if (c->pages > 0 && !c->data) return DG_ERR_INVALID_ARG;
  if (!aligned(c->data, 16)) return DG_ERR_MISALIGNED;
  return DG_OK;
}

dg_status run_rows(const dg_kv4_cache* c, int64_t tokens, uint16_t* K, int64_t ldk, uint16_t* V, int64_t ldv,
                   const int64_t* slots, void* stream, bool append) {
  const dg_status st = check_cache(c);
  if (st != DG_OK) return st;
  if (tokens < 0) return DG_ERR_INVALID_ARG;
  if (tokens == 0) return DG_OK;
  const int64_t width = static_cast<int64_t>(c->heads) * c->d;
  if (!K || !V || !slots || ldk < width || ldv < width) return DG_ERR_INVALID_ARG;
  if (tokens > INT32_MAX) return DG_ERR_UNSUPPORTED;
  if (!aligned(K, 2) || !aligned(V, 2) || !aligned(slots, 8)) return DG_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  int sms = 0;
  if (serving_device(&status, &sms) != cudaSuccess) return DG_ERR_CUDA;
  Kv4Params p;
  p.data = c->data; p.pages = c->pages; p.page_size = c->page_size; p.heads = c->heads;
  p.tokens = tokens; p.slots = slots;
  p.K = K; p.ldk = ldk; p.V = V; p.ldv = ldv;
  p.index_word = status + 1;
  const int n = c->d == 128 ? 8 : 4;  // elements of one access
  const bool vec = aligned(K, 2 * n) && aligned(V, 2 * n) && ldk % n == 0 && ldv % n == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(append ? launch_kv4_append(p, c->d, vec, sms, s) : launch_kv4_gather(p, c->d, vec, sms, s));
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status rmsnorm_residual_bf16(int64_t rows, int64_t cols, const void* X, int64_t ldx, dg_out x_type,
                                const void* R, int64_t ldr, dg_out r_type, void* H, int64_t ldh,
                                const uint16_t* gain, float eps, uint16_t* Y, int64_t ldy, void* stream) {
  const dg_status st = check_norm(rows, cols, X, ldx, x_type, R, ldr, r_type, H, ldh, gain, eps, Y, ldy);
  if (st != DG_OK || rows == 0 || cols == 0) return st;
  if (!aligned(Y, 2)) return DG_ERR_MISALIGNED;
  return run_norm(rows, cols, X, ldx, x_type, R, ldr, r_type, H, ldh, gain, eps, Y, ldy, nullptr, stream);
}

dg_status rmsnorm_residual_e4m3(int64_t rows, int64_t cols, const void* X, int64_t ldx, dg_out x_type,
                                const void* R, int64_t ldr, dg_out r_type, void* H, int64_t ldh,
                                const uint16_t* gain, float eps, uint8_t* Q, int64_t ldq, float* scales,
                                void* stream) {
  const dg_status st = check_norm(rows, cols, X, ldx, x_type, R, ldr, r_type, H, ldh, gain, eps, Q, ldq);
  if (st != DG_OK || rows == 0 || cols == 0) return st;
  if (!scales) return DG_ERR_INVALID_ARG;
  if (!aligned(scales, 4)) return DG_ERR_MISALIGNED;
  return run_norm(rows, cols, X, ldx, x_type, R, ldr, r_type, H, ldh, gain, eps, Q, ldq, scales, stream);
}

int64_t dg_kv4_block_bytes(int32_t page_size, int32_t d) {
  if (page_size <= 0 || page_size > kMaxPage || page_size % kKv4Tokens != 0 || (d != 64 && d != 128)) return 0;
  return static_cast<int64_t>(page_size / kKv4Tokens) * kv4_record_bytes(d);
}

dg_status kv4_append(const dg_kv4_cache* cache, int64_t tokens, const uint16_t* K, int64_t ldk, const uint16_t* V,
                     int64_t ldv, const int64_t* slots, void* stream) {
  return run_rows(cache, tokens, const_cast<uint16_t*>(K), ldk, const_cast<uint16_t*>(V), ldv, slots, stream, true);
}

dg_status kv4_gather(const dg_kv4_cache* cache, int64_t tokens, const int64_t* slots, uint16_t* K, int64_t ldk,
                     uint16_t* V, int64_t ldv, void* stream) {
  return run_rows(cache, tokens, K, ldk, V, ldv, slots, stream, false);
}

int64_t dg_attention_kv4_workspace_bytes(int64_t batch, int64_t Lq, int64_t heads_q, int64_t heads_kv, int32_t d) {
  if (batch <= 0 || Lq <= 0 || heads_q <= 0 || heads_kv <= 0 || heads_q % heads_kv != 0 || (d != 64 && d != 128))
    return 0;
  if (heads_kv > kMaxCacheHeads || !attention_takes(batch, Lq, heads_q)) return 0;
  return kv4_attention_ws_bytes(Lq, heads_q, heads_kv, d);
}

dg_status attention_kv4(const dg_kv4_cache* cache, int64_t batch, int64_t Lq, int64_t heads_q, float scale,
                        const uint16_t* Q, int64_t ldq, int64_t strideQ, const int32_t* page_table, int64_t ldt,
                        const int32_t* lens, uint16_t* O, int64_t ldo, int64_t strideO, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  const dg_status st = check_cache(cache);
  if (st != DG_OK) return st;
  if (batch < 0 || Lq < 0 || heads_q < 0 || ldt < 0) return DG_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return DG_ERR_INVALID_ARG;
  if (batch == 0 || Lq == 0 || heads_q == 0) return DG_OK;
  if (heads_q % cache->heads != 0) return DG_ERR_INVALID_ARG;
  if (!attention_takes(batch, Lq, heads_q) || ldt > (int64_t(1) << 28) / cache->page_size) return DG_ERR_UNSUPPORTED;
  // The kernel counts units of 32 keys of all (sequence, head, 8 query rows) in 31 bits.
  if (batch * cache->heads * ((Lq * (heads_q / cache->heads) + 7) / 8) > INT32_MAX / (ldt * cache->page_size / 32 + 1))
    return DG_ERR_UNSUPPORTED;
  const int d = cache->d;
  const int64_t width = heads_q * d;
  if (!Q || !O || !lens || (ldt > 0 && !page_table)) return DG_ERR_INVALID_ARG;
  if ((Lq > 1 && (ldq < width || ldo < width)) ||
      (batch > 1 && (!rows_fit(Lq, ldq, width, strideQ) || !rows_fit(Lq, ldo, width, strideO))))
    return DG_ERR_INVALID_ARG;
  const int64_t need = kv4_attention_ws_bytes(Lq, heads_q, cache->heads, d);
  if (!workspace || workspace_bytes < need) return DG_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(O, 16) || ldq % 8 || ldo % 8 || strideQ % 8 || strideO % 8 ||
      !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(workspace, 256))
    return DG_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  int sms = 0;
  if (serving_device(&status, &sms) != cudaSuccess) return DG_ERR_CUDA;
  Kv4AttnParams p;
  p.data = cache->data; p.pages = cache->pages; p.page_size = cache->page_size; p.heads = cache->heads;
  // floor(2^32 / d) + 1 divides exactly while n * d < 2^32: n < 2^24 records, d <= 256.
  p.page_magic = cache->page_size == kKv4Tokens
                     ? 0
                     : static_cast<uint32_t>((int64_t(1) << 32) / (cache->page_size / kKv4Tokens) + 1);
  p.batch = batch; p.Lq = Lq;
  p.group = static_cast<int32_t>(heads_q / cache->heads);
  p.c_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // log2(e)
  p.Q = Q; p.ldq = ldq; p.strideQ = strideQ;
  p.table = page_table; p.ldt = ldt; p.lens = lens;
  p.O = O; p.ldo = ldo; p.strideO = strideO;
  p.ws = workspace;
  p.status = status;
  p.index_word = status + 1;
  return from_cuda(launch_kv4_attention(p, d, sms, static_cast<cudaStream_t>(stream)));
}

int64_t dg_moe_workspace_bytes(int64_t T, int64_t K, int64_t I, int64_t E, int64_t top) {
  if (T <= 0 || K <= 0 || I <= 0 || E <= 0 || top <= 0 || top > E || !moe_takes(T, K, I, E, top)) return 0;
  return moe_ws_bytes(T, I, top);
}

dg_status moe_bf16(int64_t T, int64_t K, int64_t I, int64_t E, int64_t top, int32_t renorm, const uint16_t* X,
                   int64_t ldx, const float* logits, int64_t ldl, const uint16_t* Wg, int64_t ldwg,
                   int64_t strideWg, const uint16_t* Wu, int64_t ldwu, int64_t strideWu, const uint16_t* Wd,
                   int64_t ldwd, int64_t strideWd, uint16_t* Y, int64_t ldy, void* workspace,
                   int64_t workspace_bytes, void* stream) {
  if (T < 0 || K < 0 || I < 0 || E <= 0 || top <= 0 || top > E) return DG_ERR_INVALID_ARG;
  if (T == 0 || K == 0) return DG_OK;
  if (I == 0) return DG_ERR_INVALID_ARG;
  if (!moe_takes(T, K, I, E, top)) return DG_ERR_UNSUPPORTED;
  if (!X || !logits || !Wg || !Wu || !Wd || !Y) return DG_ERR_INVALID_ARG;
  if (ldx < K || ldl < E || ldwg < I || ldwu < I || ldwd < K || ldy < K) return DG_ERR_INVALID_ARG;
  if (E > 1 && (strideWg / K < ldwg || strideWu / K < ldwu || strideWd / I < ldwd)) return DG_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < moe_ws_bytes(T, I, top)) return DG_ERR_INVALID_ARG;
  if (!aligned(X, 16) || !aligned(Wg, 16) || !aligned(Wu, 16) || !aligned(Wd, 16) || ldx % 8 || ldwg % 8 ||
      ldwu % 8 || ldwd % 8 || strideWg % 8 || strideWu % 8 || strideWd % 8 || !aligned(logits, 4) ||
      !aligned(Y, 2) || !aligned(workspace, 256))
    return DG_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  int sms = 0;
  if (serving_device(&status, &sms) != cudaSuccess) return DG_ERR_CUDA;
  MoeParams p;
  p.T = T; p.K = K; p.I = I; p.E = E;
  p.top = static_cast<int32_t>(top);
  p.renorm = renorm != 0;
  p.X = X; p.ldx = ldx; p.logits = logits; p.ldl = ldl;
  p.Wg = Wg; p.ldwg = ldwg; p.strideWg = strideWg;
  p.Wu = Wu; p.ldwu = ldwu; p.strideWu = strideWu;
  p.Wd = Wd; p.ldwd = ldwd; p.strideWd = strideWd;
  p.Y = Y; p.ldy = ldy;
  p.ws = workspace;
  p.status = status;
  return from_cuda(launch_moe(p, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
