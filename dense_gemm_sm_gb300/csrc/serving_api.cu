// serving_api.cu -- the C ABI of the serving operators: argument checks and launches.  Every
// check that needs no GPU comes before the first CUDA call, so a refused call enqueues nothing
// and touches no device.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dg_internal.h"
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
constexpr int64_t kMaxNodes = 64;    // of a tree of drafted tokens
constexpr int64_t kMaxW4Dim = int64_t(1) << 30;  // sizes of a 4-bit weight

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

// attention_kv4 and, where `mask` is given, attention_kv4_tree (Lq <= 64).
dg_status run_attention(const dg_kv4_cache* cache, int64_t batch, int64_t Lq, int64_t heads_q, float scale,
                        const uint16_t* Q, int64_t ldq, int64_t strideQ, const int32_t* page_table, int64_t ldt,
                        const int32_t* lens, const int32_t* nodes, const uint64_t* mask, uint16_t* O, int64_t ldo,
                        int64_t strideO, void* workspace, int64_t workspace_bytes, void* stream) {
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
      !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(nodes, 4) || !aligned(mask, 8) || !aligned(workspace, 256))
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
  p.nodes = nodes;
  p.mask = mask;
  return from_cuda(launch_kv4_attention(p, d, sms, static_cast<cudaStream_t>(stream)));
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

bool is_group(int32_t group) { return group == 32 || group == 64 || group == 128; }

// The weight itself: codes of N rows, `ldq` bytes apart, and parameters of its groups, `ldp` words apart.
dg_status check_w4(int64_t N, int64_t K, int32_t group, const void* Q, int64_t ldq, const void* params, int64_t ldp) {
  if (group <= 0 || ldq < 0 || ldq / 4 < (K + 7) / 8 || ldp < N || !Q || !params) return DG_ERR_INVALID_ARG;
  if (!is_group(group) || N > kMaxW4Dim || K > kMaxW4Dim) return DG_ERR_UNSUPPORTED;
  if (!aligned(Q, 16) || ldq % 16 || !aligned(params, 16) || ldp % 4) return DG_ERR_MISALIGNED;
  return DG_OK;
}

dg_status run_w4_rows(int64_t N, int64_t K, int32_t group, uint16_t* W, int64_t ldw, uint8_t* Q, int64_t ldq,
                      uint32_t* params, int64_t ldp, void* stream, bool quantize) {
  if (N < 0 || K < 0) return DG_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return DG_OK;
  if (!W || ldw < K) return DG_ERR_INVALID_ARG;
  const dg_status st = check_w4(N, K, group, Q, ldq, params, ldp);
  if (st != DG_OK) return st;
  if (!aligned(W, 2)) return DG_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  int sms = 0;
  if (serving_device(&status, &sms) != cudaSuccess) return DG_ERR_CUDA;
  W4RowsParams p;
  p.N = N; p.K = K;
  p.W = W; p.ldw = ldw; p.Q = Q; p.ldq = ldq; p.params = params; p.ldp = ldp;
  const bool vec = aligned(W, 16) && ldw % 8 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(quantize ? launch_quantize_w4(p, group, vec, sms, s) : launch_dequantize_w4(p, group, vec, sms, s));
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
  return run_attention(cache, batch, Lq, heads_q, scale, Q, ldq, strideQ, page_table, ldt, lens, nullptr, nullptr, O, ldo,
                       strideO, workspace, workspace_bytes, stream);
}

dg_status attention_kv4_tree(const dg_kv4_cache* cache, int64_t batch, int64_t Lq, int64_t heads_q, float scale,
                             const uint16_t* Q, int64_t ldq, int64_t strideQ, const int32_t* page_table, int64_t ldt,
                             const int32_t* lens, const int32_t* nodes, const uint64_t* mask, uint16_t* O, int64_t ldo,
                             int64_t strideO, void* workspace, int64_t workspace_bytes, void* stream) {
  const dg_status st = check_cache(cache);
  if (st != DG_OK) return st;
  if (Lq > kMaxNodes) return DG_ERR_UNSUPPORTED;
  if (batch > 0 && Lq > 0 && heads_q > 0 && !mask) return DG_ERR_INVALID_ARG;
  return run_attention(cache, batch, Lq, heads_q, scale, Q, ldq, strideQ, page_table, ldt, lens, nodes, mask, O, ldo,
                       strideO, workspace, workspace_bytes, stream);
}

dg_status kv4_accept(const dg_kv4_cache* cache, int64_t batch, int64_t Lq, const int32_t* page_table, int64_t ldt,
                     const int32_t* lens, const int32_t* nodes, const int32_t* path, int64_t ldp, const int32_t* counts,
                     int32_t* new_lens, void* stream) {
  const dg_status st = check_cache(cache);
  if (st != DG_OK) return st;
  if (batch < 0 || Lq < 0 || ldt < 0) return DG_ERR_INVALID_ARG;
  if (batch == 0) return DG_OK;
  if (!lens || !counts || !new_lens || (ldt > 0 && !page_table) || (Lq > 0 && (!path || (batch > 1 && ldp < Lq))))
    return DG_ERR_INVALID_ARG;
  if (batch > kMaxAttn || Lq > kMaxNodes || ldt > (int64_t(1) << 28) / cache->page_size) return DG_ERR_UNSUPPORTED;
  if (!aligned(page_table, 4) || !aligned(lens, 4) || !aligned(nodes, 4) || !aligned(path, 4) || !aligned(counts, 4) ||
      !aligned(new_lens, 4))
    return DG_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  int sms = 0;
  if (serving_device(&status, &sms) != cudaSuccess) return DG_ERR_CUDA;
  Kv4AcceptParams p;
  p.data = cache->data; p.pages = cache->pages; p.page_size = cache->page_size; p.heads = cache->heads;
  p.batch = batch; p.Lq = static_cast<int32_t>(Lq);
  p.table = page_table; p.ldt = ldt; p.lens = lens; p.nodes = nodes;
  p.path = path; p.ldp = ldp; p.counts = counts; p.new_lens = new_lens;
  p.index_word = status + 1;
  return from_cuda(launch_kv4_accept(p, cache->d, static_cast<cudaStream_t>(stream)));
}

dg_status kv4_copy_pages(const dg_kv4_cache* cache, int64_t n, const int32_t* src, const int32_t* dst, void* stream) {
  const dg_status st = check_cache(cache);
  if (st != DG_OK) return st;
  if (n < 0) return DG_ERR_INVALID_ARG;
  if (n == 0) return DG_OK;
  if (!src || !dst) return DG_ERR_INVALID_ARG;
  if (n > INT32_MAX) return DG_ERR_UNSUPPORTED;
  if (!aligned(src, 4) || !aligned(dst, 4)) return DG_ERR_MISALIGNED;
  uint32_t* status = nullptr;
  int sms = 0;
  if (serving_device(&status, &sms) != cudaSuccess) return DG_ERR_CUDA;
  Kv4CopyParams p;
  p.data = cache->data; p.pages = cache->pages;
  p.page_bytes = dg_kv4_block_bytes(cache->page_size, cache->d) * cache->heads;
  p.n = n; p.src = src; p.dst = dst;
  p.index_word = status + 1;
  return from_cuda(launch_kv4_copy_pages(p, sms, static_cast<cudaStream_t>(stream)));
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

dg_status quantize_groups_w4(int64_t N, int64_t K, int32_t group, const uint16_t* W, int64_t ldw, uint8_t* Q,
                             int64_t ldq, uint32_t* params, int64_t ldp, void* stream) {
  return run_w4_rows(N, K, group, const_cast<uint16_t*>(W), ldw, Q, ldq, params, ldp, stream, true);
}

dg_status dequantize_groups_w4(int64_t N, int64_t K, int32_t group, const uint8_t* Q, int64_t ldq,
                               const uint32_t* params, int64_t ldp, uint16_t* W, int64_t ldw, void* stream) {
  return run_w4_rows(N, K, group, W, ldw, const_cast<uint8_t*>(Q), ldq, const_cast<uint32_t*>(params), ldp, stream, false);
}

int64_t dg_gemm_w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxW4Dim || N > kMaxW4Dim || K > kMaxW4Dim) return 0;
  return gemm_w4_ws_bytes(M, N, K);
}

dg_status gemm_w4_bf16(int64_t M, int64_t N, int64_t K, int32_t group, const uint16_t* X, int64_t ldx, const uint8_t* Q,
                       int64_t ldq, const uint32_t* params, int64_t ldp, void* C, int64_t ldc, dg_out c_type,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !is_type(c_type)) return DG_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return DG_OK;
  if (!C || ldc < N) return DG_ERR_INVALID_ARG;
  if (M > kMaxW4Dim || N > kMaxW4Dim || K > kMaxW4Dim) return DG_ERR_UNSUPPORTED;
  const bool f32 = c_type == DG_OUT_F32;
  if (K > 0) {
    if (!X || ldx < K) return DG_ERR_INVALID_ARG;
    const dg_status st = check_w4(N, K, group, Q, ldq, params, ldp);
    if (st != DG_OK) return st;
    const int64_t need = gemm_w4_ws_bytes(M, N, K);
    if (need == 0) return DG_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < need) return DG_ERR_INVALID_ARG;
    if (!aligned(X, 16) || ldx % 8 || !aligned(workspace, 256)) return DG_ERR_MISALIGNED;
  }
  if (!aligned(C, f32 ? 4 : 2)) return DG_ERR_MISALIGNED;
  if (K == 0) return from_cuda(launch_scale(C, f32, M, N, ldc, 0, 1, 0.f, static_cast<cudaStream_t>(stream)));
  uint32_t* status = nullptr;
  int sms = 0;
  if (serving_device(&status, &sms) != cudaSuccess) return DG_ERR_CUDA;
  W4GemmParams p;
  p.M = M; p.N = N; p.K = K; p.group = group; p.c_f32 = f32;
  p.X = X; p.ldx = ldx; p.Q = Q; p.ldq = ldq; p.params = params; p.ldp = ldp;
  p.C = C; p.ldc = ldc;
  p.ws = workspace;
  p.status = status;
  return from_cuda(launch_gemm_w4(p, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
