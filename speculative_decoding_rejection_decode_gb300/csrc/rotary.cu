// Dense rows turned by positions on up to four axes (images, videos), or back by the
// same (the gradient of a turn).  Contract in include/specdec.h (specdec_rotate).
//
//   a' = a cos - b sin, b' = b cos + a sin,
// cos and sin of a pair from the table's row at the position on the pair's own axis;
// products and sum rounded one by one in 32 bits, as append does, then once to the type.
// Bound by memory: a thread holds both halves of its pairs, so that nothing crosses
// lanes, and a block's cos and sin come to shared memory once for all of its heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/specdec.h"
#include "cache.cuh"
#include "row_values.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;
// Blocks of an SM: 64 registers for both halves of the pairs, fewer are wanted for
// neighbours.  50k rows of 32 heads of 64, us at 4, 5, 6 blocks: halves 70, 84, 99,
// interleaved 75, 72, 75 (410 MB: 5.8 and 5.7 TB/s).
template <bool INTERLEAVED>
constexpr int kBlocks = INTERLEAVED ? 5 : 4;
constexpr int kMaxRows = 16;   // rows of a block at most
constexpr int kU = 4;          // items of a thread under way together

__device__ __forceinline__ Vec8 turned(const Vec8& a, const Vec8& b, const float* c, const float* s, float sign) {
  Vec8 y;
#pragma unroll
  for (int k = 0; k < 8; ++k) y.x[k] = __fadd_rn(__fmul_rn(a.x[k], c[k]), sign * __fmul_rn(b.x[k], s[k]));
  return y;
}

// An item: 8 pairs (halves layout: 8 values of both halves) or 8 values that stay
// (interleaved: 8 neighbouring values either way).
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kBlocks<INTERLEAVED>) rotate_kernel(const RotateArgs a, const int rows) {
  __shared__ __align__(16) float cs[kMaxRows][kMaxPairs], sn[kMaxRows][kMaxPairs];
  __shared__ int64_t at_axis[kMaxRows][kMaxAxes];
  __shared__ int lost[kMaxRows];
  const int64_t r0 = (int64_t)blockIdx.x * rows;
  const int here = (int)min((int64_t)rows, a.N - r0), half = a.rotary_dim / 2;
  if ((int)threadIdx.x < here) {
    int bad = 0;
    for (int i = 0; i < a.num_axes; ++i) {
      const int64_t at = a.pos[i * a.pos_stride + r0 + threadIdx.x];
      if (at < 0 || at >= a.positions) bad = 1;
      at_axis[threadIdx.x][i] = at * a.rotary_dim;
    }
    lost[threadIdx.x] = bad;
    if (bad) atomicOr(a.err, SPECDEC_DEVERR_BAD_CACHE);
  }
  __syncthreads();
  const float way = a.inverse ? -1.0f : 1.0f;
  for (int x = threadIdx.x; x < here * half; x += kThreads) {
    const int i = x / half, j = x - i * half;
    if (lost[i]) continue;
    const float* from = a.rotary + at_axis[i][axis_of(a.axes, j)] + j;
    cs[i][j] = __ldg(from);
    sn[i][j] = way * __ldg(from + half);
  }
  __syncthreads();
  // A thread keeps its items of a row (where one lies takes divisions) and goes over the
  // block's rows with them, or over every `abreast`-th where a row has few.
  const int turning = INTERLEAVED ? a.rotary_dim / 8 : a.rotary_dim / 16;
  const int pieces = turning + (a.head_dim - a.rotary_dim) / 8;   // items of a head
  const int per = a.heads * pieces, abreast = per < kThreads ? kThreads / per : 1;
  const int first = per < kThreads ? (int)threadIdx.x / per : 0;
  if (first >= abreast) return;
  for (int item = (int)threadIdx.x - first * per; item < per; item += kThreads) {
    const int h = item / pieces, piece = item - h * pieces;
    const bool turns = piece < turning;
    const int d = turns ? piece * 8 : a.rotary_dim + (piece - turning) * 8;
    const T* src = static_cast<const T*>(a.x) + r0 * a.x_row + h * a.x_head + d;
    T* dst = static_cast<T*>(a.out) + r0 * a.out_row + h * a.out_head + d;
    const bool pair = !INTERLEAVED && turns;
    for (int i0 = first; i0 < here; i0 += kU * abreast) {
      uint4 lo[kU], hi[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = i0 + u * abreast;
        lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
        if (i < here && !lost[i]) {
          lo[u] = *reinterpret_cast<const uint4*>(src + i * a.x_row);
          if (pair) hi[u] = *reinterpret_cast<const uint4*>(src + i * a.x_row + half);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = i0 + u * abreast;
        if (i >= here) continue;
        uint4* out = reinterpret_cast<uint4*>(dst + i * a.out_row);
        if (!turns || lost[i]) {                  // as it is; a lost row is zeros
          *out = lo[u];
          if (pair) *reinterpret_cast<uint4*>(dst + i * a.out_row + half) = hi[u];
        } else if constexpr (INTERLEAVED) {
          const float4 c = *reinterpret_cast<const float4*>(&cs[i][piece * 4]);
          const float4 s = *reinterpret_cast<const float4*>(&sn[i][piece * 4]);
          const float* cc = &c.x;
          const float* ss = &s.x;
          const Vec8 x = widen<T>(lo[u]);
          Vec8 y;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y.x[2 * k] = __fsub_rn(__fmul_rn(x.x[2 * k], cc[k]), __fmul_rn(x.x[2 * k + 1], ss[k]));
            y.x[2 * k + 1] = __fadd_rn(__fmul_rn(x.x[2 * k + 1], cc[k]), __fmul_rn(x.x[2 * k], ss[k]));
          }
          *out = narrow<T>(y);
        } else {
          float4 c[2], s[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            c[k] = *reinterpret_cast<const float4*>(&cs[i][piece * 8 + 4 * k]);
            s[k] = *reinterpret_cast<const float4*>(&sn[i][piece * 8 + 4 * k]);
          }
          const Vec8 x = widen<T>(lo[u]), z = widen<T>(hi[u]);
          *out = narrow<T>(turned(x, z, &c[0].x, &s[0].x, -1.0f));
          *reinterpret_cast<uint4*>(dst + i * a.out_row + half) = narrow<T>(turned(z, x, &c[0].x, &s[0].x, 1.0f));
        }
      }
    }
  }
}

template <typename T>
int rotate_of(const RotateArgs& a, int num_sms, cudaStream_t st) {
  // whole waves of resident blocks, of no more rows than a block's tables hold
  const int64_t blocks = (int64_t)num_sms * (a.interleaved ? kBlocks<true> : kBlocks<false>), waves = (a.N + blocks * kMaxRows - 1) / (blocks * kMaxRows);
  int64_t rows = (a.N + blocks * waves - 1) / (blocks * waves);
  if (rows < 1) rows = 1;
  const unsigned grid = (unsigned)((a.N + rows - 1) / rows);
  if (a.interleaved) rotate_kernel<T, true><<<grid, kThreads, 0, st>>>(a, (int)rows);
  else rotate_kernel<T, false><<<grid, kThreads, 0, st>>>(a, (int)rows);
  return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace

int launch_rotate(const RotateArgs& a, int dtype, int num_sms, cudaStream_t st) {
  if (a.N == 0) return SPECDEC_OK;
  return dtype == SPECDEC_BF16 ? rotate_of<__nv_bfloat16>(a, num_sms, st) : rotate_of<__half>(a, num_sms, st);
}

}  // namespace specdec
