// The paged key/value cache: writing drafted nodes (rotary positions and 8-bit
// quantisation on the way), reading rows back, and moving an accepted branch
// into place.  Contract in include/specdec.h.
//
// Bounds: the read-back and the append by memory traffic (64 contexts of up to 8191 e4m3
// rows of 8 heads of 128 read: 1.70 GB in 258 us, 6.6 TB/s; 40619 rows of 48 heads turned
// and quantised: 918 MB in 160 us, 5.7 TB/s); the commit, and every call for one request, by
// latency (29 nodes of 48 heads written: 5 us).
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
constexpr int kAppendBlocks = 5;   // of an append on an SM

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 values / scale rounded to e4m3 (to nearest, ties to even), 8 bytes for each half.  The
// quotients are those of an IEEE division, so that the stored byte and scale are a function
// of the row alone, whatever computes them: q + (x - q scale) r is the quotient rounded to
// nearest where r is the reciprocal so rounded and q = x r (Markstein, 1990; that the bytes
// are a division's has been counted over every scale's mantissa beside every border between
// two bytes).  Taken as q - (q scale - x) r, a zero keeps its sign.  |x / scale| passes 448
// by rounding at most, which rounds back to 448.
__device__ __forceinline__ void quantise(float* x, float scale, uint2* to) {
  uint32_t w[8];
  float d = scale;
  if (!(scale < 1e30f)) {                    // out of the reciprocal's range: both by 2^-40
    d = scale == INFINITY ? 0.0f : scale * 9.094947017729282e-13f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= 9.094947017729282e-13f;
  }
  const float r = scale == INFINITY ? 0.0f : __frcp_rn(d);   // finite / inf is 0, inf / inf NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 f = make_float2(__fmul_rn(x[2 * i], r), __fmul_rn(x[2 * i + 1], r));
    f.x = __fmaf_rn(-__fmaf_rn(f.x, d, -x[2 * i]), r, f.x);
    f.y = __fmaf_rn(-__fmaf_rn(f.y, d, -x[2 * i + 1]), r, f.y);
    w[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  to[0] = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  to[1] = make_uint2(w[4] | w[5] << 16, w[6] | w[7] << 16);
}

constexpr int kRows = 24;   // rows of an append's block at most (a lane finds the place of one)
constexpr int kReadRows = 16;   // of a read's

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

// A thread has two chunks of 8 values of a row, both halves of the same pairs in the halves
// layout, so that a turn crosses no lanes; D / 16 lanes hold a row.  cos and sin of the
// block's rows, each pair's from the row of the table at the position on its own axis,
// come to shared memory all at once.  Products and their sum are rounded one by one (no
// fused multiply-add), as the formula
//   a' = a cos - b sin, b' = b cos + a sin
// reads in 32 bits, so that what is quantised does not depend on contraction.
template <typename T, bool FP8, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kAppendBlocks) append_kernel(const AppendArgs a, const int rows) {
  constexpr int LANES = D / 16;                // lanes of a row
  constexpr int SLOTS = kThreads / LANES;      // heads in flight
  __shared__ RowPlace places[kRows];
  __shared__ __align__(16) float turns[kRows][2][D / 2];   // cos, sin of a row's pairs
  __shared__ int64_t at_axis[kRows][kMaxAxes];             // their positions in the table
  const int l = threadIdx.x % LANES, slot0 = threadIdx.x / LANES;
  const CacheArgs& c = a.c;
  const int half = a.rotary_dim / 2;
  const int64_t r0 = (int64_t)blockIdx.x * rows;
  const int here = (int)min((int64_t)rows, c.N - r0);
  if (threadIdx.x < 32) {
    const int from = warp_request_of_row(c.cu, c.B, r0);
    if ((int)threadIdx.x < here) {
      const bool given = a.pos != nullptr;
      RowPlace p = place_of(c, from, r0 + threadIdx.x, !given && a.rotary != nullptr, a.rotary_dim, a.positions, a.offsets);
      if (given && p.owned) {
        p.turn = 0;
        for (int i = 0; i < a.num_axes; ++i) {
          const int64_t at = a.pos[i * a.pos_stride + r0 + threadIdx.x];
          if (at < 0 || at >= a.positions) p.row = p.turn = -1;
          at_axis[threadIdx.x][i] = at * a.rotary_dim;
        }
        if (p.turn < 0) atomicOr(c.err, SPECDEC_DEVERR_BAD_CACHE);
      } else {
        at_axis[threadIdx.x][0] = p.turn;      // (axes are all 0 here)
      }
      places[threadIdx.x] = p;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && (int64_t)c.cu[c.B] > c.N) atomicOr(c.err, SPECDEC_DEVERR_BAD_CU);
  __syncthreads();
  // this thread's chunks: their first values, and where they turn the first of their pairs
  const int pairs = INTERLEAVED ? 0 : half / 8;   // lanes that hold both halves of 8 pairs
  const bool both = l < pairs;
  const int da = both ? l * 8 : INTERLEAVED ? l * 8 : a.rotary_dim + (l - pairs) * 16;
  const int db = both ? half + l * 8 : INTERLEAVED ? (l + LANES) * 8 : da + 8;
  const int kv = c.geo.kv_heads, heads = a.q ? a.q_heads : 0;
  // A step is SLOTS heads: of k and v, one sequence of 2 kv, or of q.  The first steps' places
  // are kept from row to row, and their loads for the next row are under way while this
  // one's values are turned and stored.
  struct Values {
    uint4 a, b;
  };
  struct Lane {
    const T* from;        // this row's chunk a
    int64_t stride;
    bool on;
  };
  auto kv_lane = [&](int step) -> Lane {
    const int hh = step * SLOTS + slot0;
    if (hh < kv) return {static_cast<const T*>(a.k) + r0 * a.k_row + hh * a.k_head + da, a.k_row, true};
    return {static_cast<const T*>(a.v) + r0 * a.v_row + (hh - kv) * a.v_head + da, a.v_row, hh < 2 * kv};
  };
  auto q_lane = [&](int step) -> Lane {
    const int h = step * SLOTS + slot0;
    return {static_cast<const T*>(a.q) + r0 * a.q_row + h * a.q_head + da, a.q_row, h < heads};
  };
  const int apart = db - da;
  auto load = [&](const Lane& x, int i) -> Values {
    Values v = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (x.on && i < here && places[i].owned) {
      const T* from = x.from + i * x.stride;
      v.a = *reinterpret_cast<const uint4*>(from);    // (q may be turned in place)
      v.b = *reinterpret_cast<const uint4*>(from + apart);
    }
    return v;
  };
  float cs[8], sn[8];
  bool ta = false, tb = false;                 // whether the chunks turn
  auto turned = [&](const Values& w, bool turns_too, float* x) {
    const Vec8 va = widen<T>(w.a), vb = widen<T>(w.b);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const Vec8& v = z ? vb : va;
        const bool turn = turns_too && (z ? tb : ta);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float u = v.x[2 * k], y = v.x[2 * k + 1], cc = cs[4 * z + k], ss = sn[4 * z + k];
          x[8 * z + 2 * k] = turn ? __fsub_rn(__fmul_rn(u, cc), __fmul_rn(y, ss)) : u;
          x[8 * z + 2 * k + 1] = turn ? __fadd_rn(__fmul_rn(y, cc), __fmul_rn(u, ss)) : y;
        }
      }
    } else if (turns_too && ta) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = __fsub_rn(__fmul_rn(va.x[k], cs[k]), __fmul_rn(vb.x[k], sn[k]));
        x[8 + k] = __fadd_rn(__fmul_rn(vb.x[k], cs[k]), __fmul_rn(va.x[k], sn[k]));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = va.x[k];
        x[8 + k] = vb.x[k];
      }
    }
  };
  auto store16 = [&](T* to, const float* x) {
    *reinterpret_cast<uint4*>(to + da) = make_uint4(pack(x[0], x[1], T()), pack(x[2], x[3], T()), pack(x[4], x[5], T()), pack(x[6], x[7], T()));
    *reinterpret_cast<uint4*>(to + db) = make_uint4(pack(x[8], x[9], T()), pack(x[10], x[11], T()), pack(x[12], x[13], T()), pack(x[14], x[15], T()));
  };
  auto store_kv = [&](const Values& w, int step, const RowPlace& p) {   // the whole block calls
    const int hh = step * SLOTS + slot0;
    const bool isv = hh >= kv;
    float x[16];
    turned(w, !isv, x);
    const bool live = hh < 2 * kv && p.row >= 0;
    const int64_t row = p.row + (int64_t)((isv ? hh - kv : hh) * c.geo.page_size);
    if constexpr (FP8) {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) m = max_nan(m, fabsf(x[k]));
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (!live) return;
      const float scale = __fmul_rn(max_nan(m, kScaleFloor), 1.0f / kE4M3Max);
      uint8_t* to = static_cast<uint8_t*>(isv ? c.v : c.k) + row * D;
      uint2 bytes[2];
      quantise(x, scale, bytes);
      *reinterpret_cast<uint2*>(to + da) = bytes[0];
      *reinterpret_cast<uint2*>(to + db) = bytes[1];
      if (l == 0) (isv ? c.vs : c.ks)[row] = scale;
    } else if (live) {
      store16(static_cast<T*>(isv ? c.v : c.k) + row * D, x);
    }
  };
  auto store_q = [&](const Values& w, int step, int64_t r, bool lost) {
    const int h = step * SLOTS + slot0;
    if (h >= heads) return;
    float x[16];
    turned(w, true, x);
    if (lost) {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = 0.0f;
    }
    store16(static_cast<T*>(a.out_q) + (r * heads + h) * D, x);
  };
  const int kv_steps = (2 * kv + SLOTS - 1) / SLOTS, q_steps = (heads + SLOTS - 1) / SLOTS;
  const Lane lkv = kv_lane(0), lq0 = q_lane(0), lq1 = q_lane(1);
  Values wkv = load(lkv, 0), wq0 = load(lq0, 0), wq1 = load(lq1, 0);
  for (int x = threadIdx.x; x < here * half; x += kThreads) {
    const int i = x / half, j = x - i * half;
    if (places[i].turn < 0) continue;
    const float* from = a.rotary + at_axis[i][axis_of(a.axes, j)] + j;
    turns[i][0][j] = __ldg(from);
    turns[i][1][j] = __ldg(from + half);
  }
  __syncthreads();
  for (int i = 0; i < here; ++i) {
    const RowPlace p = places[i];
    const int64_t r = r0 + i;
    ta = tb = false;
    if (p.turn >= 0) {
      const float *cosp = turns[i][0], *sinp = turns[i][1];
      if constexpr (INTERLEAVED) {
        ta = da < a.rotary_dim;
        tb = db < a.rotary_dim;
        if (ta) {
          *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(cosp + da / 2);
          *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(sinp + da / 2);
        }
        if (tb) {
          *reinterpret_cast<float4*>(cs + 4) = *reinterpret_cast<const float4*>(cosp + db / 2);
          *reinterpret_cast<float4*>(sn + 4) = *reinterpret_cast<const float4*>(sinp + db / 2);
        }
      } else if (both) {
        ta = true;
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          *reinterpret_cast<float4*>(cs + k) = *reinterpret_cast<const float4*>(cosp + da + k);
          *reinterpret_cast<float4*>(sn + k) = *reinterpret_cast<const float4*>(sinp + da + k);
        }
      }
    }
    const bool lost = a.rotary && p.turn < 0;   // no position: defined rows
    const Values now = wkv;
    wkv = load(lkv, i + 1);
    if (p.owned) {
      store_kv(now, 0, p);
#pragma unroll 1
      for (int s = 1; s < kv_steps; ++s) store_kv(load(kv_lane(s), i), s, p);
    }
    if (heads) {
      const Values now0 = wq0;
      wq0 = load(lq0, i + 1);
      if (p.owned) store_q(now0, 0, r, lost);
      const Values now1 = wq1;
      wq1 = load(lq1, i + 1);
      if (p.owned) {
        store_q(now1, 1, r, lost);
#pragma unroll 1
        for (int s = 2; s < q_steps; ++s) store_q(load(q_lane(s), i), s, r, lost);
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
  __shared__ RowPlace places[kReadRows];
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

// Rows of an append's block, whose places are looked up together (a few dependent loads):
// as many that the blocks fill whole waves of the resident ones.  40619 rows of 48 heads
// into e4m3, 16, 24, 32 rows at most: 162, 160, 159 us, 15k (read back) 90, 88, 88; one
// wave, or 16 rows whatever is left for the last wave, 167 and 104.  Wide rows of 16 bits are
// bound by memory even within a wave, and two waves cover each other's starts: 15k of 128, 8,
// 16, 24 rows at most 64.0, 62.9, 66.6 us (without a turn 60.4, 61.3, 73.7), 16k 67.6, 67.3,
// 72.5; of 64 values 42.6, 40.4, 38.2.
template <bool FP8, int D>
constexpr int kMostRows = !FP8 && D == 128 ? 16 : kRows;

inline int rows_per_block(int64_t N, int64_t blocks, int most) {
  const int64_t waves = (N + blocks * most - 1) / (blocks * most), r = (N + blocks * waves - 1) / (blocks * waves);
  return (int)(r < 1 ? 1 : r);
}

template <typename T, bool FP8, int D>
int append_dim(const AppendArgs& a, int num_sms, cudaStream_t st) {
  const int rows = rows_per_block(a.c.N, (int64_t)num_sms * kAppendBlocks, kMostRows<FP8, D>);
  const unsigned grid = (unsigned)((a.c.N + rows - 1) / rows);
  if (a.interleaved) append_kernel<T, FP8, D, true><<<grid, kThreads, 0, st>>>(a, rows);
  else append_kernel<T, FP8, D, false><<<grid, kThreads, 0, st>>>(a, rows);
  return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

template <typename T, bool FP8>
int append_of(const AppendArgs& a, int num_sms, cudaStream_t st) {
  return a.c.head_dim == 128 ? append_dim<T, FP8, 128>(a, num_sms, st) : append_dim<T, FP8, 64>(a, num_sms, st);
}

template <typename T, bool FP8>
int read_of(const ReadArgs& a, int num_sms, cudaStream_t st) {
  const int64_t even = (a.c.N + (int64_t)num_sms * 5 - 1) / ((int64_t)num_sms * 5);   // one wave, where that is
  const int rows = (int)(even > kReadRows ? kReadRows : even);
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
