// serving.h -- shared declarations of the serving operators: residual RMS norm, the paged
// 4-bit key-value cache with its attention, and the mixture-of-experts layer.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/dgemm.h"

namespace dg {

// Status words and SM count of the current device (cached per device): status[0] is the
// bounded-wait word, status[1] the index word (a page, slot or length outside its table).
cudaError_t serving_device(uint32_t** status, int* sms);

// Value a kernel writes into the index word.
constexpr uint32_t kDevBadIndex = 0x201;

// ------------------------------------------------------------------ residual RMS norm
struct NormParams {
  int64_t rows, cols;
  const void* X; int64_t ldx;
  const void* R; int64_t ldr;   // residual in (null: none)
  void* H; int64_t ldh;         // residual out, R's type
  const uint16_t* gain;         // BF16 [cols]
  float eps;
  void* Y; int64_t ldy;         // BF16, or E4M3 codes when scales != null
  float* scales;                // [rows] (E4M3 output)
};
// x_f32 / r_f32: the types of X and of R and H.  vec: every row 16-byte aligned.
cudaError_t launch_rmsnorm(const NormParams& p, bool x_f32, bool r_f32, bool vec, cudaStream_t s);

// ------------------------------------------------------------------ 4-bit key-value cache
// Record of 16 tokens of one (page, head), bytes: K codes [16][d/2]; V codes [2][8][4][d/32][2][2]
// (token / 8, column group of d/8, token % 8 / 2, four columns, token % 2, two bytes); K
// parameters [16] words, V parameters [16] words (scale BF16 low half, zero BF16 high half).
constexpr int kKv4Tokens = 16;  // tokens of a record
constexpr __host__ __device__ int kv4_record_bytes(int d) { return kKv4Tokens * (d + 8); }

struct Kv4Params {
  uint8_t* data;
  int64_t pages;
  int32_t page_size, heads;
  int64_t tokens;
  const int64_t* slots;
  uint16_t* K; int64_t ldk;
  uint16_t* V; int64_t ldv;
  uint32_t* index_word;
};
// vec: rows of K and V aligned for 16-byte (d = 128) or 8-byte (d = 64) accesses.
cudaError_t launch_kv4_append(const Kv4Params& p, int d, bool vec, int sms, cudaStream_t s);
cudaError_t launch_kv4_gather(const Kv4Params& p, int d, bool vec, int sms, cudaStream_t s);

struct Kv4AttnParams {
  const uint8_t* data;
  int64_t pages;
  int32_t page_size, heads;         // heads: of the cache
  uint32_t page_magic;              // n / (page_size / 16) = n * magic >> 32 for n < 2^24; 0: one record a page
  int32_t one_copy;                 // set at launch: pages hold whole units
  int32_t fault;                    // set at launch: 1: stages are not released (test hook)
  int64_t batch, Lq;
  int32_t group;                    // query heads per cache head
  float c_log2;                     // scale * log2(e)
  const uint16_t* Q; int64_t ldq, strideQ;
  const int32_t* table; int64_t ldt;
  const int32_t* lens;
  uint16_t* O; int64_t ldo, strideO;
  void* ws;
  uint32_t* status;
  uint32_t* index_word;
};
int64_t kv4_attention_ws_bytes(int64_t Lq, int64_t heads_q, int64_t heads_kv, int d);
cudaError_t launch_kv4_attention(const Kv4AttnParams& p, int d, int sms, cudaStream_t s);

// ------------------------------------------------------------------ mixture of experts
struct MoeParams {
  int64_t T, K, I, E;
  int32_t top;
  int32_t renorm;
  const uint16_t* X; int64_t ldx;
  const float* logits; int64_t ldl;
  const uint16_t* Wg; int64_t ldwg, strideWg;
  const uint16_t* Wu; int64_t ldwu, strideWu;
  const uint16_t* Wd; int64_t ldwd, strideWd;
  uint16_t* Y; int64_t ldy;
  void* ws;
  uint32_t* status;
  // Set by launch_moe: CTAs on neighbouring column tiles; 1: stages are not released (test hook).
  uint32_t up_group, down_group;
  int32_t fault;
};
int64_t moe_ws_bytes(int64_t T, int64_t I, int64_t top);
cudaError_t launch_moe(const MoeParams& p, int sms, cudaStream_t s);

}  // namespace dg
