// The paged key/value cache (cache.cu), attention over it (attention.cu) and
// verification from given numbers (given.cu): arguments and launchers, shared
// with the entry points in specdec.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_index.h"

namespace specdec {

constexpr int kMaxTreeNodes = 1024;  // nodes of a request with parents that attention masks
constexpr float kE4M3Max = 448.0f;
constexpr float kScaleFloor = 9.094947017729282e-13f;  // 2^-40: least magnitude a scale stands for

struct CacheArgs {
  void* k;              // [num_pages, kv_heads, page_size, head_dim]
  void* v;
  float* ks;            // [num_pages, kv_heads, page_size], or null for 16-bit caches
  float* vs;
  PagedGeo geo;
  int head_dim;         // 64 or 128
  const int32_t* table; // [B, max_pages]
  const int32_t* lengths;  // [B]
  const int32_t* cu;       // [B + 1]
  const int32_t* parent;   // [N] or null (chains)
  int B;
  int64_t N;
  uint32_t* err;        // sticky device error word
};

struct AppendArgs {
  CacheArgs c;
  const void* k;        // [N, kv_heads, head_dim], strides in elements
  const void* v;
  const void* q;        // [N, q_heads, head_dim] or null
  int64_t k_row, k_head, v_row, v_head, q_row, q_head;
  int q_heads;
  void* out_q;          // contiguous
  const float* rotary;  // [positions, 2, rotary_dim / 2] or null
  int rotary_dim;
  int64_t positions;
  int interleaved;
};

struct ReadArgs {
  CacheArgs c;          // lengths: first slot of each request
  void* out_k;          // [N, kv_heads, head_dim]
  void* out_v;
};

struct CommitArgs {
  CacheArgs c;
  const int32_t* accepted;  // [B]
  const int32_t* path;      // [N] or null (chains)
  int32_t* out_lengths;     // [B], may be c.lengths
};

struct AttendArgs {
  CacheArgs c;
  const void* q;        // [N, q_heads, head_dim]
  int64_t q_row, q_head;
  int q_heads;
  float scale_log2;     // softmax scale * log2(e)
  void* out;            // [N, q_heads, head_dim] contiguous
  void* workspace;
  int item_cost;        // units of an item's own (attention.cuh; set by launch_attend)
  bool whole;           // items are not split: no workspace, no join (set by launch_attend)
};

struct GivenArgs {
  const float* p;       // [N_t, V], rows p_row apart
  const float* q;       // [N_d, V] or null
  int64_t p_row, q_row;
  const int32_t* ids;
  const int32_t* cu;
  const float* accept_u;
  const float* sample_u;
  int B, V;
  int64_t N_d;
  int32_t* out_tokens;
  int32_t* out_nacc;
  uint32_t* err;
  int vec_ok;           // rows are 16-byte aligned
};

// Each queues its kernels on st and returns SPECDEC_OK or SPECDEC_ERR_CUDA.
// cache_dtype, dtype: SPECDEC_BF16, SPECDEC_F16 or (cache_dtype) SPECDEC_E4M3.
int launch_append(const AppendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st);
int launch_read(const ReadArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st);
int launch_commit(const CommitArgs& a, int cache_dtype, cudaStream_t st);
int launch_attend(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st);
int64_t attend_workspace_bytes(int B, int64_t N, int kv_heads, int q_heads, int head_dim, int64_t capacity, int num_sms);
int launch_given(const GivenArgs& a, int num_sms, cudaStream_t st);

}  // namespace specdec
