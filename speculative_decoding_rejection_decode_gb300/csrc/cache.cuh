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

constexpr int kMaxAxes = 4;    // position axes of rotary pairs
constexpr int kMaxPairs = 64;  // rotary pairs of a head

// The axis of each pair, two bits a pair.
struct RotaryAxes {
  uint32_t word[kMaxPairs / 16];
};

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
  // positions of the rows' own, [num_axes, N], axes pos_stride apart, or null: length +
  // depth (+ the request's offset, where offsets is not null)
  const int32_t* pos;
  int64_t pos_stride;
  int num_axes;
  RotaryAxes axes;
  const int32_t* offsets;  // [B]
};

// Dense rows turned by positions of their own.
struct RotateArgs {
  const void* x;        // [N, heads, head_dim], strides in elements
  void* out;            // the same; may be x itself
  int64_t x_row, x_head, out_row, out_head;
  int64_t N;
  int heads, head_dim;
  const int32_t* pos;   // [num_axes, N], axes pos_stride apart
  int64_t pos_stride;
  int num_axes;
  RotaryAxes axes;
  const float* rotary;  // [positions, 2, rotary_dim / 2]
  int rotary_dim;
  int64_t positions;
  int interleaved, inverse;
  uint32_t* err;
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
  bool cross;           // the keys are the context alone
  const uint8_t* mask;  // [B, mask_slots], rows mask_stride apart, 0: hidden (cross), or null
  int64_t mask_stride, mask_slots;
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
int launch_rotate(const RotateArgs& a, int dtype, int num_sms, cudaStream_t st);
int launch_read(const ReadArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st);
int launch_commit(const CommitArgs& a, int cache_dtype, cudaStream_t st);
int launch_attend(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st);
int64_t attend_workspace_bytes(bool cross, int cache_dtype, int page_size, int B, int64_t N, int kv_heads, int q_heads, int head_dim, int64_t capacity, int num_sms);
int launch_given(const GivenArgs& a, int num_sms, cudaStream_t st);

}  // namespace specdec
