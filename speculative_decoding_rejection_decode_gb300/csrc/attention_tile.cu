// The tile kernel (attention_tile.cuh) over a request's context and its nodes.
#include "attention_tile.cuh"

namespace specdec {

int64_t attend_tile_workspace(int head_dim, int num_sms) {
  return head_dim == 128 ? Partials<kR, 128>::bytes(num_sms) : Partials<kR, 64>::bytes(num_sms);
}

int launch_attend_tile(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st) {
  return launch_tile_types<false>(a, cache_dtype, dtype, num_sms, st);
}

}  // namespace specdec
