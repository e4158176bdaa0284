// Log probabilities of given tokens with entropy and top alternatives, and the
// gradient of the logits (logprob.cu): arguments and launchers, shared with the entry
// points in specdec.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace specdec {

constexpr int kMaxTop = 32;   // alternatives of a token at most

struct LogprobArgs {
  const void* x;            // [R, V] logits, rows row_stride elements apart
  int64_t row_stride, R;
  int V;
  float c;                  // log2(e) / T
  const int32_t* ids;       // [M] or null
  const int32_t* rows;      // [M] or null (token t's row is t)
  int64_t M;
  int top;
  float* logprob;           // [M], or null
  float* entropy;           // [M], or null
  int32_t* top_ids;         // [M, top]
  float* top_logprobs;      // [M, top]
  float2* stats;            // [M] (reference logit, log2 of the sum), or null
  uint32_t* err;
};

struct LogprobGradArgs {
  const void* x;            // [M, V]
  int64_t row_stride, M;
  int V;
  float c, inv_t;
  const int32_t* ids;       // [M] or null
  int top;
  const float* logprob;     // what the forward call gave
  const float* entropy;
  const int32_t* top_ids;
  const float* top_logprobs;
  const float2* stats;
  const float* g_logprob;   // [M] or null, each
  const float* g_entropy;
  const float* g_top;       // [M, top]
  void* out;                // [M, V], rows out_stride apart; may be x
  int64_t out_stride;
};

int launch_logprob(const LogprobArgs& a, int dtype, int num_sms, cudaStream_t st);
int launch_logprob_grad(const LogprobGradArgs& a, int dtype, int num_sms, cudaStream_t st);

}  // namespace specdec
