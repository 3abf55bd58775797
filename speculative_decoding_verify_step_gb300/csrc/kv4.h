// Host-side launchers of the 4-bit paged KV cache (kv4.cu, kv4_attention.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace spec {

// Where flat row r of a call lies in the pool.  Either row_slot gives its physical
// slot (page * 64 + offset, or < 0: none), or the row's sequence and position do:
// sequence b owns rows row_off[b] .. row_off[b + 1] - 1 (row_off null: rows_per_seq
// each) at positions start[b] + 0, 1, ... of page table row b.
struct Kv4Rows {
  const int32_t* row_slot;
  const int32_t* row_off;
  const int32_t* start;
  const int32_t* page_table;
  int B, rows_per_seq, max_pages, num_pages;
  int total_rows;
};

struct Kv4WriteParams {
  Kv4Rows rows;
  int Hkv, hd, bf16;
  const void* k;
  const void* v;
  // element offset of (row r, head h): (r / row_blk) * blk_stride + (r % row_blk) * row_stride + h * head_stride
  int row_blk;
  long long blk_stride, k_row_stride, v_row_stride, head_stride;
  uint8_t* pool;
};
// Pseudo-random cells (the hash of the fp16 cache's fill) on every page of the listed sequences,
// all layers; layer l's pool is pool + l * layer_bytes.
cudaError_t launch_kv4_fill_pages(uint8_t* pool, long long layer_bytes, const int32_t* page_table,
                                  const int32_t* seq_npages, int max_pages, const int32_t* seq_ids, int n, int n_layers,
                                  int num_pages, int Hkv, int hd, uint64_t seed, float scale, cudaStream_t st);
cudaError_t launch_kv4_write(const Kv4WriteParams& p, cudaStream_t st);

struct Kv4ReadParams {
  Kv4Rows rows;
  int Hkv, hd, bf16;
  void* k;
  void* v;  // [total_rows, Hkv, hd]
  const uint8_t* pool;
};
cudaError_t launch_kv4_read(const Kv4ReadParams& p, cudaStream_t st);

struct Kv4AttnParams {
  const void* q;               // row r at q + r * q_row_stride, [Hq, hd]
  long long q_row_stride;
  void* out;                   // [total_rows, Hq, hd]
  int bf16;
  const uint8_t* pool;
  const int32_t* page_table;   // row of sequence b: b, or seq_ids[b]
  const int32_t* seq_ids;      // null: b
  const int32_t* kv_len;       // [B] cached tokens before the window
  const int32_t* row_begin;    // [B] (or [B + 1]) first flat row of sequence b; null: b * W
  const int32_t* row_count;    // [B] rows of sequence b; null: row_begin[b + 1] - row_begin[b], or W
  int B, W, total_rows, Hq, Hkv, hd;
  int max_pages, num_pages, table_rows;
  int sm_count, kv_len_hint;   // launch shape only
  float scale;                 // of q . k
  float scale_m, scale_2;      // |scale| log2(e) as a mantissa in [1, 2) (or 0) times a power of two: set by the launcher
  uint32_t anc[16];            // window rows that row j sees (bit i)
  // Inside a model's forward: the cached pages and the sequence state were complete
  // before the predecessor let this kernel launch, so only q and the window's K/V
  // are waited for.  0: everything is.
  int early;
  int stages, slots, cluster;  // ring depth, CTAs resident at once, CTAs of a cluster: set by the launcher
  float* workspace;            // kv4_attention_workspace bytes
  // Weights of the projections that follow, brought into L2 once the queries are
  // there; split evenly over the CTAs.  Null / 0: none.
  const void* l2_next[2];
  unsigned long long l2_next_bytes[2];  // multiples of 16
  int* status;
};
// Bytes of workspace for windows of `rows` query rows per kv head (W * group size).
long long kv4_attention_workspace(int B, int Hkv, int rows, int hd, int kv_len_hint, int sm_count);
cudaError_t launch_kv4_attention(const Kv4AttnParams& p, cudaStream_t st);

}  // namespace spec
