// The tile kernel (attention_tile.cuh) over an encoder's states.
#include "attention_tile.cuh"

namespace specdec {

int launch_cross_tile(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st) {
  return launch_tile_types<true>(a, cache_dtype, dtype, num_sms, st);
}

}  // namespace specdec
