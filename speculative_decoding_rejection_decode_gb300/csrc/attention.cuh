// Attention of drafted nodes over the paged cache: what its kernels share.
//
// Work is a flat list of units: for every request, kv head and row tile (an
// item), one unit per tile of keys.  The units are split into as many equal
// contiguous ranges as there are CTAs, so that ragged lengths leave no CTA
// idle; an item that crosses a range leaves partial results (row maximum, sum
// and weighted sum of values) that a second, dependent kernel joins.
//
// An item also counts item_cost units of its own: starting and ending it (queries,
// an empty pipeline, results) takes about as long as that many tiles, and without
// them the ranges that hold many short requests finished late.  us at a cost of 2, 4,
// 5, 6 (32 query and 8 kv heads of 128): tile kernel, 64 requests of 2 to 9 nodes over up
// to 8191 keys, bf16 237, 221, 219, 216; 32 of 29 over 6000 to 16000, e4m3 303, 298, 296,
// 296; warp kernel at a cost of 1, 2, 3, 5, 64 of 1 over up to 8191, bf16 193, 183, 180,
// 180; 200 of 1 to 4 over up to 1500, bf16 182, 170, 157, 151; 64 of 2 to 9 over up to
// 2047, 32 kv heads, bf16 300, 256, 236, 216 (at 7 and more it rises again); e4m3 at 2, 3,
// 4, 6: 178, 183, 185, 191; 173, 179, 183, 191; 258, 259, 269, 286 (its tiles are of 256
// keys and take longer).
//
// Rows of an item: r = node * group + head within the group, so one read of a
// key serves every node and every query head that shares it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/specdec.h"
#include "cache.cuh"
#include "device_common.cuh"

namespace specdec {

constexpr int kItemCost = 5;       // units of an item's own
constexpr int kItemCostWarp8 = 2;  // the same in the warp kernel over 8-bit caches

struct Request {
  int64_t first;   // first node row
  int64_t units;
  int32_t n;       // nodes
  int32_t len;     // context
  int32_t rts;     // row tiles
  int32_t tiles;   // key tiles
};

// What the plan of a call depends on.
struct PlanArgs {
  const int32_t* cu;
  const int32_t* lengths;
  int64_t N, capacity;      // node rows; slots of a request
  int32_t B, kv_heads, group, item_cost;
  bool tree, whole, cross;  // whole: items are not split; cross: the keys are the context alone

  __host__ __device__ __forceinline__ explicit PlanArgs(const AttendArgs& a)
      : cu(a.c.cu), lengths(a.c.lengths), N(a.c.N), capacity((int64_t)a.c.geo.max_pages * a.c.geo.page_size), B(a.c.B),
        kv_heads(a.c.geo.kv_heads), group(a.q_heads / a.c.geo.kv_heads), item_cost(a.item_cost), tree(a.c.parent != nullptr), whole(a.whole), cross(a.cross) {}
};

// Whether a call leaves items whole: contexts of at most 4 tiles by the page
// table's width, and no more items than two for each CTA.  One launch and no
// workspace then; splitting such items only pays where they are many and ragged.
// Device us, whole and split, 32 query and 8 kv heads of 128, bf16: 1 request of 1 node
// over 60 / 250 / 480 keys 7.5 and 8.9 / 9.3 and 10.9 / 11.6 and 11.0 (a call,
// host included: 17.0 and 23.2, for the second launch and the workspace), of 29 nodes 12.3 and 15.6 /
// 14.0 and 20.0 / 15.7 and 20.8; 32 requests of 1 node 12.3 and 13.8 / 15.8 and 19.8 /
// 23.0 and 27.3, of 29 nodes 21.2 and 26.0 / 31.1 and 40.0 / 36.4 and 46.2.
inline bool whole_items(int B, int64_t N, int kv_heads, int q_heads, int64_t capacity, int rows, int num_sms) {
  const int64_t avg = (N + B - 1) / B * (q_heads / kv_heads);
  return capacity <= 512 && (int64_t)B * kv_heads * ((avg + rows - 1) / rows) <= 2 * (int64_t)num_sms;
}

// The plan of request b for tiles of R rows and TK keys.  units = 0 for what
// cannot be attended (no nodes, a cu or length out of range, a tree that is
// too large); why gets the error bits.
__host__ __device__ __forceinline__ Request attend_request(const PlanArgs& c, int b, int R, int TK, uint32_t& why) {
  Request q = {};
  if (!node_range(c.cu, b, c.N, q.first, q.n)) {
    why |= SPECDEC_DEVERR_BAD_CU;
    return q;
  }
  q.len = c.lengths[b];
  if (q.n == 0) return q;
  const int64_t keys = (int64_t)q.len + (c.cross ? 0 : q.n);
  if (q.len < 0 || keys > c.capacity) {
    why |= SPECDEC_DEVERR_BAD_CACHE;
    return q;
  }
  if (c.tree && q.n > kMaxTreeNodes) {
    why |= SPECDEC_DEVERR_BAD_TREE;
    return q;
  }
  q.rts = (int32_t)(((int64_t)q.n * c.group + R - 1) / R);
  q.tiles = (int32_t)((keys + TK - 1) / TK);
  if (q.tiles == 0) q.tiles = 1;   // no key at all: rows of zeros are still to be written
  q.units = (int64_t)c.kv_heads * q.rts * ((c.whole ? 1 : q.tiles) + c.item_cost);
  if (q.units >= ((int64_t)1 << 31)) {   // units of a request are counted in 32 bits
    q.units = 0;
    why |= SPECDEC_DEVERR_BAD_CACHE;
  }
  return q;
}

#ifdef __CUDACC__

struct ScanShared {
  int64_t warp[32];
  int64_t total;
  int64_t before;
  int32_t b;
};

// Units of all requests, and the request that holds unit `want(total)` with
// the units before it.  Every thread of the block calls; NT threads.
template <int NT, typename Want>
__device__ __forceinline__ void find_unit(const PlanArgs& c, int R, int TK, Want want,
                                          ScanShared& sh, uint32_t& why) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (c.B + NT - 1) / NT;
  const int b0 = min(c.B, tid * per), b1 = min(c.B, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += attend_request(c, b, R, TK, why).units;
  int64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += up;
  }
  if (lane == 31) sh.warp[warp] = scan;
  if (tid == 0) sh.b = -1;
  __syncthreads();
  if (tid == 0) {
    int64_t t = 0;
    for (int w = 0; w < NT / 32; ++w) {
      const int64_t x = sh.warp[w];
      sh.warp[w] = t;
      t += x;
    }
    sh.total = t;
  }
  __syncthreads();
  const int64_t u = want(sh.total);
  int64_t at = sh.warp[warp] + scan - mine;
  if (at <= u && u < at + mine) {   // one thread at most
    for (int b = b0; b < b1; ++b) {
      const int64_t x = attend_request(c, b, R, TK, why).units;
      if (u < at + x) {
        sh.b = b;
        sh.before = at;
        break;
      }
      at += x;
    }
  }
  __syncthreads();
}

// Ancestors (with itself) of node j as bits of `words` words; a parent that is
// no earlier node ends the walk (false).
__device__ __forceinline__ bool ancestor_bits(const int32_t* parent, int j, int words, uint32_t* bits) {
  for (int w = 0; w < words; ++w) bits[w] = 0;
  while (true) {
    bits[j >> 5] |= 1u << (j & 31);
    if (j == 0) return true;
    const int up = parent[j];
    if (up < 0 || up >= j) return false;
    j = up;
  }
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(float x, __half& y) { y = __float2half_rn(x); }

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// The sum that marks a row whose node's parents do not lead to node 0 (sums are at
// least 0, or NaN): any part of an item that meets the break gives it, and the row
// becomes zeros.
constexpr float kLostRow = -INFINITY;

// Workspace: two partial slots per range, each R rows of D sums, then (max, sum).
// A range may go on with an item that began earlier (slot 0) and leave another to
// the next range (slot 1).
template <int R, int D>
struct Partials {
  float* sums;
  float2* stats;
  __host__ __device__ Partials(void* ws, int G)   // from a multiple of 32 bytes: rows are stored 32 at a time
      : sums(reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws) + 31) & ~(uintptr_t)31)),
        stats(reinterpret_cast<float2*>(sums + (int64_t)2 * G * R * D)) {}
  static constexpr int64_t bytes(int G) { return (int64_t)2 * G * R * (D * 4 + 8) + 32; }
};

// Joins the partial results of the items that several ranges share.  An item
// whose first tile is in range i - 1 and that goes on into range i belongs to blocks (i, *);
// block (i, y) takes 8 of its rows, a warp two of them.
template <typename T, int R, int TK, int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const AttendArgs a, const int G) {
  __shared__ ScanShared sh;
  const int group = a.q_heads / a.c.geo.kv_heads;
  const PlanArgs plan(a);
  uint32_t why = 0;
  int64_t u = 0;
  int ranges = 0;
  find_unit<128>(plan, R, TK,
                 [&](int64_t units) {
                   ranges = (int)min((int64_t)G, units);
                   u = (int)blockIdx.x + 1 < ranges ? range_begin(units, ranges, blockIdx.x + 1) : units;
                   return u;
                 },
                 sh, why);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x + 1 >= ranges || sh.b < 0) return;
  const int g0 = blockIdx.x;                     // the range before the boundary
  const Request q = attend_request(plan, sh.b, R, TK, why);
  if (q.units == 0) return;
  const int64_t item = (u - sh.before) / (q.tiles + plan.item_cost);
  const int64_t u0 = sh.before + item * (q.tiles + plan.item_cost) + plan.item_cost, u1 = u0 + q.tiles;   // its tiles
  // not an item that begins at the boundary, nor one that range g0 also went on with
  if (u0 >= u || range_begin(sh.total, ranges, g0) > u0) return;
  const int h = (int)(item / q.rts), rt = (int)(item % q.rts);
  const int g1 = range_of(sh.total, ranges, u1 - 1);
  const Partials<R, D> part(a.workspace, G);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = q.n * group;
  constexpr int PER = D / 32;
  for (int r = blockIdx.y * 8 + warp; r < (int)blockIdx.y * 8 + 8; r += 4) {
    const int row = rt * R + r;
    if (row >= rows) break;
    // range g0 left the item in its second slot, the others began inside it
    const int64_t at0 = (2 * (int64_t)g0 + 1) * R + r;
    auto at_of = [&](int g) { return g == g0 ? at0 : 2 * (int64_t)g * R + r; };
    float m = -INFINITY;
    bool gone = false;
    for (int g = g0 + lane; g <= g1; g += 32) {
      const float2 s = part.stats[at_of(g)];
      m = fmaxf(m, s.x);
      gone |= s.y == kLostRow;
    }
    m = warp_max(m);
    gone = __any_sync(0xFFFFFFFFu, gone);
    const float ref = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, acc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = 0.0f;
    constexpr int U = 4;
    for (int g = g0; g <= g1; g += U) {      // four partials' loads under way together
      float2 s[U];
      float v[U][PER];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = make_float2(-INFINITY, 0.0f);
        if (g + u <= g1) {
          const int64_t at = at_of(g + u);
          s[u] = part.stats[at];
          const float* p = part.sums + at * D + lane * PER;
          if constexpr (PER == 4) {
            const float4 x = *reinterpret_cast<const float4*>(p);
            v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(p);
            v[u][0] = x.x; v[u][1] = x.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = ex2(s[u].x - ref);
        l += s[u].y * w;
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[k] += s[u].x == -INFINITY ? 0.0f : v[u][k] * w;
      }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T* out = static_cast<T*>(a.out) +
             ((q.first + row / group) * a.q_heads + h * group + row % group) * (int64_t)D + lane * PER;
#pragma unroll
    for (int k = 0; k < PER; k += 2)
      *reinterpret_cast<uint32_t*>(out + k) = gone ? 0u : pack2(acc[k] * inv, acc[k + 1] * inv, T());
  }
}

// Allows `kern` its dynamic shared memory on the current device, once for each
// device (`done`: one word of device bits for each kernel).
template <typename K>
bool allow_shared(K kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

// Queues the join as a dependent of the attention kernel before it.
template <typename T, int R, int TK, int D>
int launch_join(const AttendArgs& a, int G, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)G, R / 8);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<T, R, TK, D>, a, G) == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

#endif  // __CUDACC__

// The tensor-core kernel (attention_tile.cu).
int launch_attend_tile(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st);
// Both kernels over an encoder's states (cross_tile.cu, cross.cu).
int launch_cross_tile(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st);
int launch_cross_warp(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st);
// Many rows per request over 16-bit states in pages of a multiple of 8 slots (cross_wide.cu).
constexpr int kWideRows = 256;   // of an item's tile
int launch_cross_wide(const AttendArgs& a, int dtype, int num_sms, cudaStream_t st);
int64_t cross_wide_workspace(int head_dim, int num_sms);
int64_t attend_tile_workspace(int head_dim, int num_sms);


}  // namespace specdec
