// Host-side launchers of the 8-bit paged KV cache (kv8.cu, kv8_attention.cu, kv8_evict.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kv4.h"

namespace spec {

struct Kv8WriteParams {
  Kv4Rows rows;  // row_slot is not used
  int Hkv, hd, bf16;
  const void* k;
  const void* v;
  long long k_row_stride, v_row_stride;
  uint8_t* pool;
};
cudaError_t launch_kv8_write(const Kv8WriteParams& p, cudaStream_t st);

struct Kv8ReadParams {
  Kv4Rows rows;
  int Hkv, hd, bf16;
  void* k;
  void* v;  // [total_rows, Hkv, hd]
  const uint8_t* pool;
};
cudaError_t launch_kv8_read(const Kv8ReadParams& p, cudaStream_t st);

struct Kv8AttnParams {
  const void* q;               // row r at q + r * q_row_stride, [Hq, hd]
  long long q_row_stride;
  void* out;                   // [total_rows, Hq, hd]
  int bf16;
  const uint8_t* pool;
  const int32_t* page_table;
  const int32_t* kv_len;       // [B] cached tokens before the window
  const int32_t* row_off;      // [B + 1] or null: W rows each
  int B, W, total_rows, Hq, Hkv, hd;
  int max_pages, num_pages;
  int sm_count, kv_len_hint;   // launch shape only
  float scale;                 // of q . k
  uint32_t anc[16];            // window rows that row j sees (bit i)
  int slots, cluster;          // CTAs resident at once, CTAs of a cluster: set by the launcher
  float* workspace;            // kv8_attention_workspace bytes: partials, then norm and scores
  float2* norm;                // [total_rows, Hq] each row's maximum and inverse sum, or null: set by the launcher
  float* scores;               // [B, Hkv, units of 32 tokens, rows, 32] or null: set by the launcher
  float* weight;               // [B, Hkv, weight_len] or null
  long long weight_len;
  int* status;
};
// Bytes of workspace of a call of p's shape (B, W, total_rows, Hq, Hkv, hd, max_pages, sm_count,
// kv_len_hint): partials of cut groups, and with `weight` the rows' sums and perhaps their scores.
long long kv8_attention_workspace(const Kv8AttnParams& p, bool weight);
// Whether that is more than none whatever the GPU.
bool kv8_attention_needs_workspace(const Kv8AttnParams& p, bool weight);
cudaError_t launch_kv8_attention(const Kv8AttnParams& p, cudaStream_t st);

struct Kv8EvictParams {
  uint8_t* pool;
  const int32_t* kv_len;       // [B]
  const int32_t* page_table;   // [B, max_pages]
  const int32_t* dst_table;    // [B, dst_pages]
  const float* weight;         // [B, Hkv, weight_len]
  int32_t* new_len;            // [B]
  int32_t* kept;               // [B, Hkv, keep]
  float* weight_out;           // [B, Hkv, weight_out_len]
  long long weight_len, weight_out_len;
  int B, Hkv, hd, max_pages, dst_pages, num_pages, keep, recent;
};
cudaError_t launch_kv8_evict(const Kv8EvictParams& p, cudaStream_t st);

}  // namespace spec
