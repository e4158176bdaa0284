// The paged key/value cache: writing drafted nodes (rotary positions and 8-bit
// quantisation on the way), reading rows back, and moving an accepted branch
// into place.  Contract in include/specdec.h.
//
// All three are bound by memory traffic (latency for one request): a thread
// moves 8 values (16 bytes of a 16-bit row) and a row of head_dim values is
// held by head_dim / 8 neighbouring lanes, so that a row's absolute maximum is
// a few shuffles and nothing passes through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/specdec.h"
#include "cache.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 128;

struct Vec8 {
  float x[8];
};

__device__ __forceinline__ float2 unpack(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
__device__ __forceinline__ uint32_t pack(float a, float b, __nv_bfloat16) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack(float a, float b, __half) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ Vec8 widen(uint4 w) {
  Vec8 v;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack(u[i], T());
    v.x[2 * i] = f.x;
    v.x[2 * i + 1] = f.y;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ uint4 narrow(const Vec8& v) {
  return make_uint4(pack(v.x[0], v.x[1], T()), pack(v.x[2], v.x[3], T()),
                    pack(v.x[4], v.x[5], T()), pack(v.x[6], v.x[7], T()));
}

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

// 8 neighbouring cos (or sin) of the table, or 4 of them each used twice.
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// One block per row of a tile: threads are (head slot, chunk of 8 values); a
// thread keeps its cos and sin for every head it turns.  Products and their
// sum are rounded one by one (no fused multiply-add), as the formula
//   a' = a cos - b sin, b' = b cos + a sin
// reads in 32 bits, so that what is quantised does not depend on contraction.
template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a, const int rows) {
  constexpr int LANES = D / 8;                 // lanes of a row
  constexpr int SLOTS = kThreads / LANES;      // heads in flight
  const int chunk = threadIdx.x % LANES, slot0 = threadIdx.x / LANES;
  const CacheArgs& c = a.c;
  const int half = a.rotary_dim / 2;
  const int d0 = chunk * 8;
  for (int64_t r = (int64_t)blockIdx.x * rows; r < min((int64_t)(blockIdx.x + 1) * rows, c.N); ++r) {
    const int b = request_of_row(c.cu, c.B, r);
    if (b < 0) {  // rows behind the last request are not touched
      if (threadIdx.x == 0 && r < (int64_t)c.cu[c.B]) atomicOr(c.err, SPECDEC_DEVERR_BAD_CU);
      continue;
    }
    const int64_t first = c.cu[b];
    const int j = (int)(r - first);
    const int64_t len = c.lengths[b];
    const int64_t row0 = len < 0 ? -1 : cache_row(c.geo, c.table + b * c.geo.table_stride, len + j);
    bool live = row0 >= 0;
    uint32_t bad = live ? 0u : SPECDEC_DEVERR_BAD_CACHE;
    const float *cosp = nullptr, *sinp = nullptr;
    if (a.rotary) {
      const int depth = node_depth(c.parent ? c.parent + first : nullptr, j);
      const int64_t pos = len + depth;
      if (depth < 0) {
        bad |= SPECDEC_DEVERR_BAD_TREE;
        live = false;
      } else if (len < 0 || pos >= a.positions) {
        bad |= SPECDEC_DEVERR_BAD_CACHE;
        live = false;
      } else {
        cosp = a.rotary + pos * 2 * half;
        sinp = cosp + half;
      }
    }
    if (bad && threadIdx.x == 0) atomicOr(c.err, bad);
    const bool turned = cosp && d0 < a.rotary_dim;
    float cs[8], sn[8];
    int64_t partner = 0;
    float sign = 1.0f;
    if (turned) {
      if (a.interleaved) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(cosp + d0 / 2));
        const float4 y = __ldg(reinterpret_cast<const float4*>(sinp + d0 / 2));
        cs[0] = cs[1] = x.x; cs[2] = cs[3] = x.y; cs[4] = cs[5] = x.z; cs[6] = cs[7] = x.w;
        sn[0] = sn[1] = y.x; sn[2] = sn[3] = y.y; sn[4] = sn[5] = y.z; sn[6] = sn[7] = y.w;
      } else {
        const bool low = d0 < half;
        load8(cosp + (low ? d0 : d0 - half), cs);
        load8(sinp + (low ? d0 : d0 - half), sn);
        partner = low ? half : -half;
        sign = low ? -1.0f : 1.0f;
      }
    }
    const int turns = a.q ? a.q_heads : 0;
    // heads in order: k, v, then q, SLOTS at a time; every lane of a warp takes
    // part in each step, with its own source row
    const int total = 2 * c.geo.kv_heads + turns;
    for (int h0 = 0; h0 < total; h0 += SLOTS) {
      const int hh = h0 + slot0;
      const bool isk = hh < c.geo.kv_heads;
      const bool isv = !isk && hh < 2 * c.geo.kv_heads;
      const bool any = hh < total;
      const int h = isk ? hh : (isv ? hh - c.geo.kv_heads : hh - 2 * c.geo.kv_heads);
      const T* src = nullptr;
      if (any)
        src = isk ? static_cast<const T*>(a.k) + r * a.k_row + h * a.k_head
                  : isv ? static_cast<const T*>(a.v) + r * a.v_row + h * a.v_head
                        : static_cast<const T*>(a.q) + r * a.q_row + h * a.q_head;
      Vec8 x = {};
      if (any) {
        x = widen<T>(__ldg(reinterpret_cast<const uint4*>(src + d0)));
        if (turned && !isv) {
          Vec8 y;
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              y.x[i] = __fsub_rn(__fmul_rn(x.x[i], cs[i]), __fmul_rn(x.x[i + 1], sn[i]));
              y.x[i + 1] = __fadd_rn(__fmul_rn(x.x[i + 1], cs[i]), __fmul_rn(x.x[i], sn[i]));
            }
          } else {
            const Vec8 o = widen<T>(__ldg(reinterpret_cast<const uint4*>(src + d0 + partner)));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              y.x[i] = __fadd_rn(__fmul_rn(x.x[i], cs[i]), sign * __fmul_rn(o.x[i], sn[i]));
          }
          x = y;
        }
      }
      // stored rows and turned q rows part here; row_amax needs whole warps, so
      // the 8-bit store runs for every lane and q lanes drop its result
      if (FP8 && h0 < 2 * c.geo.kv_heads) {
        void* base = isk ? c.k : c.v;
        store_row<T, FP8, D>(base, isk ? c.ks : c.vs, row0 + (int64_t)h * c.geo.page_size, chunk, x,
                             any && live && (isk || isv));
      } else if (!FP8 && any && (isk || isv)) {
        store_row<T, FP8, D>(isk ? c.k : c.v, nullptr, row0 + (int64_t)h * c.geo.page_size, chunk, x, live);
      }
      if (any && !isk && !isv) {
        if (a.rotary && !cosp) x = Vec8{};  // no position: a defined row
        reinterpret_cast<uint4*>(static_cast<T*>(a.out_q) + (r * a.q_heads + h) * D)[chunk] = narrow<T>(x);
      }
    }
  }
}

template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a, const int rows) {
  constexpr int LANES = D / 8;
  constexpr int SLOTS = kThreads / LANES;
  const int chunk = threadIdx.x % LANES, slot0 = threadIdx.x / LANES;
  const CacheArgs& c = a.c;
  for (int64_t r = (int64_t)blockIdx.x * rows; r < min((int64_t)(blockIdx.x + 1) * rows, c.N); ++r) {
    const int b = request_of_row(c.cu, c.B, r);
    if (b < 0) {
      if (threadIdx.x == 0 && r < (int64_t)c.cu[c.B]) atomicOr(c.err, SPECDEC_DEVERR_BAD_CU);
      continue;
    }
    const int64_t len = c.lengths[b];
    const int64_t row0 =
        len < 0 ? -1 : cache_row(c.geo, c.table + b * c.geo.table_stride, len + (r - c.cu[b]));
    if (row0 < 0 && threadIdx.x == 0) atomicOr(c.err, SPECDEC_DEVERR_BAD_CACHE);
    for (int hh = slot0; hh < 2 * c.geo.kv_heads; hh += SLOTS) {
      const bool isk = hh < c.geo.kv_heads;
      const int h = isk ? hh : hh - c.geo.kv_heads;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (row0 >= 0) {
        const int64_t row = row0 + (int64_t)h * c.geo.page_size;
        if constexpr (FP8) {
          const uint2 e = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(isk ? c.k : c.v) + row * D) + chunk);
          const float s = __ldg((isk ? c.ks : c.vs) + row);
          Vec8 x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t half = (i < 2 ? e.x : e.y) >> ((i & 1) * 16);
            const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(half & 0xFFFFu), __NV_E4M3);
            const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&f));
            x.x[2 * i] = g.x * s;
            x.x[2 * i + 1] = g.y * s;
          }
          w = narrow<T>(x);
        } else {
          w = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(isk ? c.k : c.v) + row * D) + chunk);
        }
      }
      T* out = static_cast<T*>(isk ? a.out_k : a.out_v) + (r * c.geo.kv_heads + h) * D;
      reinterpret_cast<uint4*>(out)[chunk] = w;
    }
  }
}

// One block per request.  A thread owns 16 bytes of a head's row (or a scale)
// and moves them for d = 0, 1, ... in order.  Paths rise (path[d] > path[d-1],
// so path[d] >= d + 1): no row that is still to be read has been written.
__global__ void __launch_bounds__(256) commit_kernel(const CommitArgs a, const int row_bytes) {
  const CacheArgs& c = a.c;
  const int b = blockIdx.x;
  int64_t first;
  int32_t n;
  const int64_t len = c.lengths[b];
  __shared__ int bad;
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
  bool ok = acc >= 0 && (acc < n || (acc == 0 && n == 0));
  uint32_t why = SPECDEC_DEVERR_BAD_TREE;
  if (ok && a.path) {
    for (int d = threadIdx.x; d < acc; d += blockDim.x) {
      const int32_t at = a.path[first + d], before = d ? a.path[first + d - 1] : 0;
      if (at <= before || at >= n) bad = 1;
      else if (cache_row(c.geo, pages, len + at) < 0 || cache_row(c.geo, pages, len + d + 1) < 0) bad = 2;
    }
  }
  __syncthreads();
  if (bad) {
    ok = false;
    if (bad == 2) why = SPECDEC_DEVERR_BAD_CACHE;
  }
  if (!ok) {
    if (threadIdx.x == 0) {
      atomicOr(c.err, why);
      a.out_lengths[b] = (int32_t)len;
    }
    return;
  }
  if (threadIdx.x == 0) a.out_lengths[b] = (int32_t)(len + (n ? 1 + acc : 0));
  if (!a.path) return;
  const int vecs = row_bytes / 16, per = 2 * vecs + (c.ks ? 2 : 0);
  for (int t = threadIdx.x; t < c.geo.kv_heads * per; t += blockDim.x) {
    const int h = t / per, w = t % per;
    for (int d = 0; d < acc; ++d) {
      const int32_t at = a.path[first + d];
      if (at == d + 1) continue;
      const int64_t src = cache_row(c.geo, pages, len + at) + (int64_t)h * c.geo.page_size;
      const int64_t dst = cache_row(c.geo, pages, len + d + 1) + (int64_t)h * c.geo.page_size;
      if (w < 2 * vecs) {
        uint4* base = static_cast<uint4*>(w < vecs ? c.k : c.v);
        const int at16 = w < vecs ? w : w - vecs;
        base[dst * vecs + at16] = base[src * vecs + at16];
      } else {
        float* s = w == 2 * vecs ? c.ks : c.vs;
        s[dst] = s[src];
      }
    }
  }
}

inline int rows_per_block(int64_t N, int num_sms, int most) {
  const int64_t r = N / ((int64_t)num_sms * 16);
  return (int)(r < 1 ? 1 : (r > most ? most : r));
}

template <typename T, bool FP8>
int append_of(const AppendArgs& a, int num_sms, cudaStream_t st) {
  const int rows = rows_per_block(a.c.N, num_sms, 4);
  const int64_t grid = (a.c.N + rows - 1) / rows;
  if (a.c.head_dim == 128) append_kernel<T, FP8, 128><<<(unsigned)grid, kThreads, 0, st>>>(a, rows);
  else append_kernel<T, FP8, 64><<<(unsigned)grid, kThreads, 0, st>>>(a, rows);
  return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

template <typename T, bool FP8>
int read_of(const ReadArgs& a, int num_sms, cudaStream_t st) {
  const int rows = rows_per_block(a.c.N, num_sms, 16);
  const int64_t grid = (a.c.N + rows - 1) / rows;
  if (a.c.head_dim == 128) read_kernel<T, FP8, 128><<<(unsigned)grid, kThreads, 0, st>>>(a, rows);
  else read_kernel<T, FP8, 64><<<(unsigned)grid, kThreads, 0, st>>>(a, rows);
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

int launch_commit(const CommitArgs& a, int cache_dtype, int num_sms, cudaStream_t st) {
  (void)num_sms;
  const int row_bytes = a.c.head_dim * (cache_dtype == SPECDEC_E4M3 ? 1 : 2);
  commit_kernel<<<a.c.B, 256, 0, st>>>(a, row_bytes);
  return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace specdec
