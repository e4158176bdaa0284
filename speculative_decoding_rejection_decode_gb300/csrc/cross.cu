// The warp kernel (attention_warp.cuh) over an encoder's states.
#include "attention_warp.cuh"

namespace specdec {

int launch_cross_warp(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st) {
  return launch_warp_types<true>(a, cache_dtype, dtype, num_sms, st);
}

}  // namespace specdec
