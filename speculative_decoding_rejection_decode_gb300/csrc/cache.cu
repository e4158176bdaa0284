// The paged key/value cache: writing drafted nodes (rotary positions and 8-bit
// quantisation on the way), reading rows back, and moving an accepted branch
// into place.  Contract in include/specdec.h.
//
// A thread moves 8 values (16 bytes of a 16-bit row) and a row of head_dim values is
// held by head_dim / 8 neighbouring lanes, so that a row's absolute maximum is
// a few shuffles and nothing passes through shared memory.  Bounds: the read-back by
// memory traffic (64 contexts of up to 8191 e4m3 rows of 8 heads of 128: 1.70 GB in
// 258 us, 6.6 TB/s); the append by no single unit (65 % of the issue slots, 62 % of the
// copy rate: a block's rows follow one another, each waiting for its own loads, after
// the look-ups before the first; 15k tree nodes of 48 heads, with their read-back: 435
// MB in 95 us); the commit, and every call for one request,
// by latency (29 nodes of 48 heads written: 4.5 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/specdec.h"
#include "cache.cuh"
#include "row_values.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Absolute maximum of a row held by LANES neighbouring lanes.
template <int LANES>
__device__ __forceinline__ float row_amax(const Vec8& v) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v.x[i]));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}

// x / scale rounded to e4m3 (to nearest, ties to even).  An IEEE division: the
// stored byte and scale are a function of the row alone, whatever computes
// them.  |x / scale| passes 448 by rounding at most, which rounds back to 448.
__device__ __forceinline__ uint2 quantise(const Vec8& v, float scale) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__fdiv_rn(v.x[2 * i], scale), __fdiv_rn(v.x[2 * i + 1], scale));
    const uint32_t two = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    w[i >> 1] |= two << ((i & 1) * 16);
  }
  return make_uint2(w[0], w[1]);
}

// Writes one lane's 8 values of a cache row.  All lanes of the warp call.
template <typename T, bool FP8, int D>
__device__ __forceinline__ void store_row(void* base, float* scales, int64_t row, int chunk,
                                          const Vec8& v, bool live) {
  if constexpr (FP8) {
    const float m = row_amax<D / 8>(v);
    const float scale = __fmul_rn(max_nan(m, kScaleFloor), 1.0f / kE4M3Max);
    const uint2 w = quantise(v, scale);
    if (live) {
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + row * D)[chunk] = w;
      if (chunk == 0) scales[row] = scale;
    }
  } else {
    if (live) reinterpret_cast<uint4*>(static_cast<T*>(base) + row * D)[chunk] = narrow<T>(v);
  }
}

// 4 neighbouring cos (or sin), of the table or (SHARED) of the block's own copy, or 8.
template <bool SHARED>
__device__ __forceinline__ float4 load4(const float* p) {
  if constexpr (SHARED) return *reinterpret_cast<const float4*>(p);
  else return __ldg(reinterpret_cast<const float4*>(p));
}
template <bool SHARED>
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = load4<SHARED>(p), b = load4<SHARED>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

constexpr int kRows = 16;   // rows of a block at most

// Where the rows of a block lie: found by one thread each, all at once, before
// any value is moved.
struct RowPlace {
  int64_t row;        // cache row of head 0, -1: none
  int64_t turn;       // offset of the position's cos in the rotary table, -1: none
  int32_t owned;      // the row belongs to a request
};

// Request of a block's first row, by a warp: 32 places of cu at a time (a thread's
// bisection of 512 requests waits for 9 loads in a row).  -1: none.
__device__ __forceinline__ int warp_request_of_row(const int32_t* cu, int B, int64_t r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;          // cu[lo] <= r is looked for with the largest lo < hi
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool below = at < hi && (int64_t)__ldg(cu + at) <= r;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, below);
    const int last = who ? 31 - __clz(who) : 0;
    hi = min(hi, lo + (last + 1) * step);
    lo = lo + last * step;
  }
  return (int64_t)__ldg(cu + lo) <= r ? lo : -1;
}

// The request of row r, from that of an earlier row: the next few, or a bisection.
__device__ __forceinline__ int request_from(const int32_t* cu, int B, int b, int64_t r) {
  if (b >= 0) {
    for (int i = 0; i < 8 && b < B; ++i, ++b) {
      if ((int64_t)cu[b] > r) break;
      if (r < (int64_t)cu[b + 1]) return b;
    }
  }
  return request_of_row(cu, B, r);
}

__device__ __forceinline__ RowPlace place_of(const CacheArgs& c, int from, int64_t r, bool rotary, int rotary_dim,
                                             int64_t positions, const int32_t* offsets = nullptr) {
  RowPlace p = {-1, -1, 0};
  uint32_t bad = 0;
  const int b = request_from(c.cu, c.B, from, r);
  if (b < 0) {  // rows behind the last request are not touched
    if (r < (int64_t)c.cu[c.B]) atomicOr(c.err, SPECDEC_DEVERR_BAD_CU);
    return p;
  }
  int64_t first;
  int32_t nodes;
  if (!node_range(c.cu, b, c.N, first, nodes)) {
    atomicOr(c.err, SPECDEC_DEVERR_BAD_CU);
    return p;
  }
  p.owned = 1;
  const int64_t len = c.lengths[b];
  const int j = (int)(r - first);
  p.row = len < 0 ? -1 : cache_row(c.geo, c.table + b * c.geo.table_stride, len + j);
  if (p.row < 0) bad |= SPECDEC_DEVERR_BAD_CACHE;
  if (rotary) {
    const int depth = node_depth(c.parent ? c.parent + first : nullptr, j);
    if (depth < 0) bad |= SPECDEC_DEVERR_BAD_TREE;
    else {
      const int64_t at = len + depth + (offsets ? offsets[b] : 0);
      if (len < 0 || at < 0 || at >= positions) bad |= SPECDEC_DEVERR_BAD_CACHE;
      else p.turn = at * rotary_dim;
    }
    if (p.turn < 0) p.row = -1;
  }
  if (bad) atomicOr(c.err, bad);
  return p;
}

// Threads are (head slot, chunk of 8 values); a thread keeps its cos and sin for
// every head it turns.  Products and their sum are rounded one by one (no fused
// multiply-add), as the formula
//   a' = a cos - b sin, b' = b cos + a sin
// reads in 32 bits, so that what is quantised does not depend on contraction.
// k and v, which may be quantised, and q have loops of their own, the first with one
// copy of its body: one loop for all heads, unrolled, was 8 % slower for one tree and
// held 6 blocks of an SM where this form holds 7.
// AXES: the rows bring positions on several axes, and each pair turns by its own; the
// block then takes the cos and sin of its rows' pairs to shared memory, all at once.
template <typename T, bool FP8, int D, bool AXES>
__global__ void __launch_bounds__(kThreads, 7) append_kernel(const AppendArgs a, const int rows) {
  constexpr int LANES = D / 8;                 // lanes of a row
  constexpr int SLOTS = kThreads / LANES;      // heads in flight
  __shared__ RowPlace places[kRows];
  __shared__ __align__(16) float turns[AXES ? kRows : 1][2][AXES ? D / 2 : 4];   // cos, sin of a row's pairs
  __shared__ int64_t at_axis[AXES ? kRows : 1][kMaxAxes];                      // their positions in the table
  const int chunk = threadIdx.x % LANES, slot0 = threadIdx.x / LANES;
  const CacheArgs& c = a.c;
  const int half = a.rotary_dim / 2;
  const int d0 = chunk * 8;
  const int64_t r0 = (int64_t)blockIdx.x * rows;
  const int here = (int)min((int64_t)rows, c.N - r0);
  if (threadIdx.x < 32) {
    const int from = warp_request_of_row(c.cu, c.B, r0);
    if ((int)threadIdx.x < here) {
      RowPlace p = place_of(c, from, r0 + threadIdx.x, !AXES && a.rotary != nullptr, a.rotary_dim, a.positions, a.offsets);
      if constexpr (AXES) {
        if (p.owned) {
          p.turn = 0;
          for (int i = 0; i < a.num_axes; ++i) {
            const int64_t at = a.pos[i * a.pos_stride + r0 + threadIdx.x];
            if (at < 0 || at >= a.positions) p.row = p.turn = -1;
            at_axis[threadIdx.x][i] = at * a.rotary_dim;
          }
          if (p.turn < 0) atomicOr(c.err, SPECDEC_DEVERR_BAD_CACHE);
        }
      }
      places[threadIdx.x] = p;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && (int64_t)c.cu[c.B] > c.N) atomicOr(c.err, SPECDEC_DEVERR_BAD_CU);
  __syncthreads();
  if constexpr (AXES) {
    for (int x = threadIdx.x; x < here * half; x += kThreads) {
      const int i = x / half, j = x - i * half;
      if (places[i].turn < 0) continue;
      const float* from = a.rotary + at_axis[i][axis_of(a.axes, j)] + j;
      turns[i][0][j] = __ldg(from);
      turns[i][1][j] = __ldg(from + half);
    }
    __syncthreads();
  }
  const int kv = c.geo.kv_heads, heads = a.q ? a.q_heads : 0;
  for (int i = 0; i < here; ++i) {
    const RowPlace p = places[i];
    if (!p.owned) continue;
    const int64_t r = r0 + i;
    const bool turned = p.turn >= 0 && d0 < a.rotary_dim, half_layout = p.turn >= 0 && !a.interleaved;
    float cs[8], sn[8];
    int partner = 0;
    float sign = 1.0f;
    if (turned) {
      const float *cosp = AXES ? turns[AXES ? i : 0][0] : a.rotary + p.turn, *sinp = AXES ? turns[AXES ? i : 0][1] : cosp + half;
      if (a.interleaved) {
        const float4 x = load4<AXES>(cosp + d0 / 2);
        const float4 y = load4<AXES>(sinp + d0 / 2);
        cs[0] = cs[1] = x.x; cs[2] = cs[3] = x.y; cs[4] = cs[5] = x.z; cs[6] = cs[7] = x.w;
        sn[0] = sn[1] = y.x; sn[2] = sn[3] = y.y; sn[4] = sn[5] = y.z; sn[6] = sn[7] = y.w;
      } else {
        const bool low = d0 < half;
        load8<AXES>(cosp + (low ? d0 : d0 - half), cs);
        load8<AXES>(sinp + (low ? d0 : d0 - half), sn);
        partner = (low ? half : -half) / 8;
        sign = low ? -1.0f : 1.0f;
      }
    }
    const int other = (int)(threadIdx.x & 31 & ~(LANES - 1)) | (chunk + partner);   // lane of the pairs' other halves
    auto turn = [&](uint4 w, bool keys) -> Vec8 {   // the whole warp calls
      Vec8 x = widen<T>(w);
      uint4 o = w;
      if (half_layout) {   // the same in the whole block
        o.x = __shfl_sync(0xFFFFFFFFu, w.x, other);
        o.y = __shfl_sync(0xFFFFFFFFu, w.y, other);
        o.z = __shfl_sync(0xFFFFFFFFu, w.z, other);
        o.w = __shfl_sync(0xFFFFFFFFu, w.w, other);
      }
      if (!turned || !keys) return x;
      Vec8 y;
      if (a.interleaved) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          y.x[k] = __fsub_rn(__fmul_rn(x.x[k], cs[k]), __fmul_rn(x.x[k + 1], sn[k]));
          y.x[k + 1] = __fadd_rn(__fmul_rn(x.x[k + 1], cs[k]), __fmul_rn(x.x[k], sn[k]));
        }
      } else {
        const Vec8 z = widen<T>(o);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          y.x[k] = __fadd_rn(__fmul_rn(x.x[k], cs[k]), sign * __fmul_rn(z.x[k], sn[k]));
      }
      return y;
    };
    // k and v heads two steps of SLOTS at a time, q heads four; the first of both are
    // under way together
    constexpr int UK = 2, UQ = 4;
    const T* q0 = static_cast<const T*>(a.q) + r * a.q_row + d0;
    uint4 wq[UQ];
    auto load_q = [&](int h0) {
#pragma unroll
      for (int u = 0; u < UQ; ++u) {
        const int h = h0 + u * SLOTS + slot0;
        wq[u] = h < heads ? __ldg(reinterpret_cast<const uint4*>(q0 + h * a.q_head)) : make_uint4(0, 0, 0, 0);
      }
    };
    for (int h0 = 0; h0 < 2 * kv; h0 += UK * SLOTS) {
      uint4 w[UK];
#pragma unroll
      for (int u = 0; u < UK; ++u) {
        const int hh = h0 + u * SLOTS + slot0;
        const T* src = hh < kv ? static_cast<const T*>(a.k) + r * a.k_row + hh * a.k_head
                               : static_cast<const T*>(a.v) + r * a.v_row + (hh - kv) * a.v_head;
        w[u] = hh < 2 * kv ? __ldg(reinterpret_cast<const uint4*>(src + d0)) : make_uint4(0, 0, 0, 0);
      }
      if (h0 == 0) load_q(0);
#pragma unroll 1
      for (int u = 0; u < UK; ++u) {
        const int hh = h0 + u * SLOTS + slot0;
        const bool isk = hh < kv;
        const Vec8 x = turn(u ? w[1] : w[0], isk);
        const int64_t row = p.row + (int64_t)(isk ? hh : hh - kv) * c.geo.page_size;
        store_row<T, FP8, D>(isk ? c.k : c.v, isk ? c.ks : c.vs, row, chunk, x, hh < 2 * kv && p.row >= 0);
      }
    }
    const bool lost = a.rotary && p.turn < 0;   // no position: defined rows
    T* out0 = static_cast<T*>(a.out_q) + r * heads * D + d0;
    for (int h0 = 0; h0 < heads; h0 += UQ * SLOTS) {
      if (h0) load_q(h0);
#pragma unroll
      for (int u = 0; u < UQ; ++u) {
        const int h = h0 + u * SLOTS + slot0;
        const Vec8 x = turn(wq[u], true);
        if (h < heads) *reinterpret_cast<uint4*>(out0 + h * D) = lost ? make_uint4(0, 0, 0, 0) : narrow<T>(x);
      }
    }
  }
}

// A thread takes 16 bytes of a cache row (16 or 8 values) at a time, four under
// way together.
template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(256) read_kernel(const ReadArgs a, const int rows) {
  constexpr int CH = FP8 ? D / 16 : D / 8;     // 16-byte chunks of a cache row
  constexpr int U = 4;
  __shared__ RowPlace places[kRows];
  const CacheArgs& c = a.c;
  const int64_t r0 = (int64_t)blockIdx.x * rows;
  const int here = (int)min((int64_t)rows, c.N - r0);
  if (threadIdx.x < 32) {
    const int from = warp_request_of_row(c.cu, c.B, r0);
    if ((int)threadIdx.x < here) places[threadIdx.x] = place_of(c, from, r0 + threadIdx.x, false, 0, 0);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && (int64_t)c.cu[c.B] > c.N) atomicOr(c.err, SPECDEC_DEVERR_BAD_CU);
  __syncthreads();
  const int kv = c.geo.kv_heads, per = 2 * kv * CH, items = here * per;
  for (int i0 = threadIdx.x; i0 < items; i0 += U * 256) {
    uint4 w[U];
    float s[U];
    T* out[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256;
      out[u] = nullptr;
      w[u] = make_uint4(0, 0, 0, 0);
      s[u] = 0.0f;
      if (i >= items) continue;
      const int in = i / per, at = i - in * per, hh = at / CH, ch = at % CH;
      const RowPlace p = places[in];
      if (!p.owned) continue;
      const bool isk = hh < kv;
      const int h = isk ? hh : hh - kv;
      out[u] = static_cast<T*>(isk ? a.out_k : a.out_v) + ((r0 + in) * kv + h) * D + ch * (FP8 ? 16 : 8);
      if (p.row < 0) continue;                 // a slot that the cache does not hold: zeros
      const int64_t row = p.row + (int64_t)h * c.geo.page_size;
      w[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(isk ? c.k : c.v) + row * (CH * 16)) + ch);
      if constexpr (FP8) s[u] = __ldg((isk ? c.ks : c.vs) + row);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!out[u]) continue;
      if constexpr (FP8) {
        const uint32_t e[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          Vec8 x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t two = e[2 * z + (k >> 1)] >> ((k & 1) * 16);
            const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
            const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&f));
            x.x[2 * k] = g.x * s[u];
            x.x[2 * k + 1] = g.y * s[u];
          }
          reinterpret_cast<uint4*>(out[u])[z] = narrow<T>(x);
        }
      } else {
        *reinterpret_cast<uint4*>(out[u]) = w[u];
      }
    }
  }
}

// One block per request.  A thread owns 16 bytes of a head's row (or a scale)
// and moves them for d = 0, 1, ... in order, four under way together.  Paths rise
// (path[d] > path[d-1], so path[d] >= d + 1): no row that is still to be read has
// been written.
__global__ void __launch_bounds__(256) commit_kernel(const CommitArgs a, const int row_bytes) {
  const CacheArgs& c = a.c;
  const int b = blockIdx.x;
  int64_t first;
  int32_t n;
  const int64_t len = c.lengths[b];
  __shared__ uint32_t bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();  // every thread has read the length that thread 0 may replace
  if (!node_range(c.cu, b, c.N, first, n) || len < 0) {
    if (threadIdx.x == 0) {
      atomicOr(c.err, len < 0 ? SPECDEC_DEVERR_BAD_CACHE : SPECDEC_DEVERR_BAD_CU);
      a.out_lengths[b] = (int32_t)len;
    }
    return;
  }
  const int32_t acc = a.accepted[b];
  const int32_t* pages = c.table + b * c.geo.table_stride;
  uint32_t why = acc >= 0 && (acc < n || (acc == 0 && n == 0)) ? 0u : (uint32_t)SPECDEC_DEVERR_BAD_TREE;
  if (!why && n) {
    // the slots that the new length takes in, len .. len + acc, are the cache's own,
    // for chains too: an append may have left their rows out
    if (len + acc >= min((int64_t)c.geo.max_pages * c.geo.page_size, (int64_t)INT32_MAX)) {
      why = SPECDEC_DEVERR_BAD_CACHE;
    } else {
      for (int d = threadIdx.x; d <= acc; d += blockDim.x) {
        uint32_t found = cache_row(c.geo, pages, len + d) < 0 ? SPECDEC_DEVERR_BAD_CACHE : 0u;
        if (a.path && d < acc) {
          const int32_t at = a.path[first + d], before = d ? a.path[first + d - 1] : 0;
          if (at <= before || at >= n) found |= SPECDEC_DEVERR_BAD_TREE;
          else if (cache_row(c.geo, pages, len + at) < 0) found |= SPECDEC_DEVERR_BAD_CACHE;
        }
        if (found) atomicOr(&bad, found);
      }
    }
  }
  __syncthreads();
  why |= bad;
  if (why) {
    if (threadIdx.x == 0) {
      atomicOr(c.err, why);
      a.out_lengths[b] = (int32_t)len;
    }
    return;
  }
  if (threadIdx.x == 0) a.out_lengths[b] = (int32_t)(len + (n ? 1 + acc : 0));
  if (!a.path) return;
  const int vecs = row_bytes / 16, per = 2 * vecs + (c.ks ? 2 : 0);
  constexpr int kMoves = 64;
  __shared__ int64_t from[kMoves], to[kMoves];   // cache rows of head 0
  for (int d0 = 0; d0 < acc; d0 += kMoves) {
    const int moves = min(kMoves, acc - d0);
    __syncthreads();
    if ((int)threadIdx.x < moves) {
      const int d = d0 + threadIdx.x;
      const int32_t at = a.path[first + d];
      from[threadIdx.x] = cache_row(c.geo, pages, len + at);
      to[threadIdx.x] = cache_row(c.geo, pages, len + d + 1);
    }
    __syncthreads();
    for (int t = threadIdx.x; t < c.geo.kv_heads * per; t += blockDim.x) {
      const int h = t / per, w = t % per;
      const int64_t head = (int64_t)h * c.geo.page_size;
      constexpr int U = 4;
      for (int m0 = 0; m0 < moves; m0 += U) {
        if (w < 2 * vecs) {
          uint4* base = static_cast<uint4*>(w < vecs ? c.k : c.v) + (w < vecs ? w : w - vecs);
          uint4 x[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (m0 + u < moves) x[u] = base[(from[m0 + u] + head) * vecs];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (m0 + u < moves) base[(to[m0 + u] + head) * vecs] = x[u];
        } else {
          float* s = w == 2 * vecs ? c.ks : c.vs;
          float x[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (m0 + u < moves) x[u] = s[from[m0 + u] + head];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (m0 + u < moves) s[to[m0 + u] + head] = x[u];
        }
      }
    }
  }
}

// Rows of a block, whose places are looked up together (a few dependent loads).
// Both take one wave of resident blocks where N allows.  Appends of 48 heads and
// 15k rows in all took 94 us with their read-back, two waves 97, three 104.
inline int rows_per_block(int64_t N, int64_t blocks, int most) {
  const int64_t r = (N + blocks - 1) / blocks;
  return (int)(r < 1 ? 1 : (r > most ? most : r));
}

template <typename T, bool FP8>
int append_of(const AppendArgs& a, int num_sms, cudaStream_t st) {
  const int rows = rows_per_block(a.c.N, (int64_t)num_sms * 7, 16);
  const int64_t grid = (a.c.N + rows - 1) / rows;
  if (a.pos) {
    if (a.c.head_dim == 128) append_kernel<T, FP8, 128, true><<<(unsigned)grid, kThreads, 0, st>>>(a, rows);
    else append_kernel<T, FP8, 64, true><<<(unsigned)grid, kThreads, 0, st>>>(a, rows);
  } else {
    if (a.c.head_dim == 128) append_kernel<T, FP8, 128, false><<<(unsigned)grid, kThreads, 0, st>>>(a, rows);
    else append_kernel<T, FP8, 64, false><<<(unsigned)grid, kThreads, 0, st>>>(a, rows);
  }
  return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

template <typename T, bool FP8>
int read_of(const ReadArgs& a, int num_sms, cudaStream_t st) {
  const int rows = rows_per_block(a.c.N, (int64_t)num_sms * 5, kRows);
  const int64_t grid = (a.c.N + rows - 1) / rows;
  if (a.c.head_dim == 128) read_kernel<T, FP8, 128><<<(unsigned)grid, 256, 0, st>>>(a, rows);
  else read_kernel<T, FP8, 64><<<(unsigned)grid, 256, 0, st>>>(a, rows);
  return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace

int launch_append(const AppendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st) {
  if (a.c.N == 0) return SPECDEC_OK;
  const bool fp8 = cache_dtype == SPECDEC_E4M3;
  if (dtype == SPECDEC_BF16)
    return fp8 ? append_of<__nv_bfloat16, true>(a, num_sms, st) : append_of<__nv_bfloat16, false>(a, num_sms, st);
  return fp8 ? append_of<__half, true>(a, num_sms, st) : append_of<__half, false>(a, num_sms, st);
}

int launch_read(const ReadArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st) {
  if (a.c.N == 0) return SPECDEC_OK;
  const bool fp8 = cache_dtype == SPECDEC_E4M3;
  if (dtype == SPECDEC_BF16)
    return fp8 ? read_of<__nv_bfloat16, true>(a, num_sms, st) : read_of<__nv_bfloat16, false>(a, num_sms, st);
  return fp8 ? read_of<__half, true>(a, num_sms, st) : read_of<__half, false>(a, num_sms, st);
}

int launch_commit(const CommitArgs& a, int cache_dtype, cudaStream_t st) {
  const int row_bytes = a.c.head_dim * (cache_dtype == SPECDEC_E4M3 ? 1 : 2);
  commit_kernel<<<a.c.B, 256, 0, st>>>(a, row_bytes);
  return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace specdec
