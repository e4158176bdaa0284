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
// them the ranges that hold many short requests finished late.  us (32 query heads of 128;
// requests of rows over keys or states, 8 kv heads unless said):
//   tile, 16 bits, cost 2, 3, 5, 8: 64 of 2-9 over up to 8191 205, 189, 180, 182
//   tile, 8 bits, 5, 6, 8, 10, 12: 32 of 29 over 1500-12000 145, 145, 142, 145, 145; 64 of 2-9
//     over up to 8191 185, 176, 179, 180, 183; 200 of 5-29 over up to 1500 223, 215, 211, 211, 213;
//     32 of 29 over 6000-16000 (context and nodes) 250, 248, 247, 245, 244
//   the same over context and nodes in pages of 16, where the table holds 8192 slots at most, 5, 6,
//     7, 10: 64 of 2-9 over up to 2000 113, 115, 120, 126; 128 of 9 over up to 1000 130, 132, 138,
//     146; 16 of 29 f16 rows over up to 6000 96, 100, 101, 109 (1 of 29 over 2000 25.9, 25.5, 25.6, 24.4)
//   wide, 2, 3, 4, 5, 7: 8 of 1000-2048 over 1500-4096 391, 386, 388, 393, 401; 64 of 100-200
//     over 500-2000 241, 236, 236, 242, 241; 30 of 200-900 over 100-700 (16 kv heads of 64)
//     97, 95, 97, 99, 98
//   warp, 16 bits, 1, 2, 3, 5: 64 of 1 over up to 8191 193, 176, 177, 174; 200 of 1-4 over up to
//     1500 189, 157, 149, 145; 64 of 2-9 over up to 2047 (32 kv heads) 224, 192, 180, 174
//     (at 7 and more it rises again)
//   warp, 8 bits, 2, 3, 4, 6: 184, 187, 189, 197; 171, 180, 188, 196; 173, 176, 179, 189 (its
//     tiles are of 256 keys and take longer)
//
// Rows of an item: r = node * group + head within the group, so one read of a
// key serves every node and every query head that shares it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/specdec.h"
#include "cache.cuh"
#include "device_common.cuh"

namespace specdec {

constexpr int kItemCost = 5;       // units of an item's own
constexpr int kItemCostTile8 = 10;  // in the tile kernel over 8-bit caches
constexpr int kItemCostTile8Short = 6, kShortSlots = 8192;   // the same over context and nodes, slots of a request
constexpr int kItemCostWide = 4;    // in the wide kernel
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
// over 60 / 250 / 480 keys 7.4 and 8.4 / 9.4 and 11.1 / 11.3 and 10.9 (a call,
// host included: 17.0 and 23.2, for the second launch and the workspace), of 29 nodes 14.1 and 15.6 /
// 17.6 and 20.0 / 19.5 and 20.1; 32 requests of 1 node 11.9 and 12.9 / 15.4 and 19.5 /
// 19.3 and 24.0, of 29 nodes 22.9 and 24.2 / 28.9 and 34.6 / 34.2 and 42.0.
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

// An item that range i leaves unfinished: what the join needs of it.
struct alignas(16) OpenItem {
  int64_t first;       // node row of its request
  int64_t end, units;  // its last unit + 1; units of the call
  int32_t rows, h, rt; // rows of its request (nodes x group), kv head, row tile
  int32_t ranges;      // of the call; 0: the range leaves none
};

// Workspace: two partial slots per range, each R rows of D sums, then (max, sum); then what
// the range leaves.  A range may go on with an item that began earlier (slot 0) and leave
// another to the next range (slot 1).
template <int R, int D>
struct Partials {
  float* sums;
  float2* stats;
  OpenItem* open;
  __host__ __device__ Partials(void* ws, int G)   // from a multiple of 32 bytes: rows are stored 32 at a time
      : sums(reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws) + 31) & ~(uintptr_t)31)),
        stats(reinterpret_cast<float2*>(sums + (int64_t)2 * G * R * D)),
        open(reinterpret_cast<OpenItem*>(stats + (int64_t)2 * G * R)) {}
  static constexpr int64_t bytes(int G) { return (int64_t)2 * G * R * (D * 4 + 8) + G * (int64_t)sizeof(OpenItem) + 32; }
};

// Joins the partial results of the items that several ranges share.  What range g leaves
// unfinished belongs to blocks (g, *), of 16 rows each, a warp four of them.  No more
// than this is done behind the attention kernel, whose ranges end together: with the plan
// walked again here, and rows in turns, the join took 19 us of 207 (8-bit states, 32
// requests of 29 nodes, 1500 to 12000 states), this form 13; the warp kernel's is hidden
// by the launch where requests are many.  Few of them have their items in many ranges, each
// block alone on its SM, and then a row's partials are what takes time: 2, 4 and 8 of them
// under way, 1 row over 2000 keys 16.5, 14.2, 13.6 us, 4000 17.2, 14.1, 13.5, 8000 in e4m3
// 21.5, 18.3, 17.7, 64 of up to 8191 188.9, 187.4, 186.6.  Tiles of 128 and 256 rows want the
// blocks on an SM: 2 and 4 (4 blocks), 32 requests of 29 nodes over 6000 to 16000 in e4m3 256
// and 259, 8 prompts of 1000 to 2048 rows 415 and 420 (1 of 29 over 5000 keys 28.7 and 27.4).
template <typename T, int R, int D>
__global__ void __launch_bounds__(128, R == 16 ? 2 : 8) attend_join_kernel(const AttendArgs a, const int G) {
  constexpr int J = 4, U = R == 16 ? 8 : 2, PER = D / 32;   // rows of a warp, partials under way together
  using V = typename std::conditional<PER == 4, float4, float2>::type;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = a.q_heads / a.c.geo.kv_heads;
  const Partials<R, D> part(a.workspace, G);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const OpenItem it = part.open[blockIdx.x];
  if (it.ranges == 0) return;
  const int g0 = blockIdx.x, g1 = range_of(it.units, it.ranges, it.end - 1), r0 = (int)blockIdx.y * 16 + warp * J;
  const int live = min(J, it.rows - (it.rt * R + r0));
  if (live <= 0) return;
  // range g0 left the item in its second slot, the others began inside it
  auto at_of = [&](int g, int j) { return (2 * (int64_t)g + (g == g0 ? 1 : 0)) * R + r0 + j; };
  V v[U][J];
  auto fetch = [&](int g) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        v[u][j] = V{};
        if (g + u <= g1 && j < live) v[u][j] = *reinterpret_cast<const V*>(part.sums + at_of(g + u, j) * D + lane * PER);
      }
  };
  fetch(g0);
  // lane 8 j + p looks after row j in every eighth range
  const int mine = lane >> 3, p = lane & 7;
  auto stat = [&](int g) { return g <= g1 && mine < live ? part.stats[at_of(g, mine)] : make_float2(-INFINITY, 0.0f); };
  float m = -INFINITY, l = 0.0f, acc[J][PER];
  int gone = 0;
  for (int g = g0 + p; g <= g1; g += 8) {
    const float2 s = stat(g);
    m = fmaxf(m, s.x);
    gone |= s.y == kLostRow;
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    gone |= __shfl_xor_sync(0xFFFFFFFFu, gone, o);
  }
  if (m == -INFINITY) m = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[j][k] = 0.0f;
  for (int c = g0; c <= g1; c += 8) {
    const float2 s = stat(c + p);
    float w = ex2(s.x - m);
    l += s.y * w;
    if (s.x == -INFINITY) w = -1.0f;             // nothing there: its sums are not looked at
    for (int i = 0; i < 8 && c + i <= g1; i += U) {
      if (c + i > g0) fetch(c + i);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float by = __shfl_sync(0xFFFFFFFFu, w, j * 8 + i + u);
          const float* x = reinterpret_cast<const float*>(&v[u][j]);
#pragma unroll
          for (int k = 0; k < PER; ++k) acc[j][k] += by < 0.0f ? 0.0f : x[k] * by;
        }
    }
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  const float inv_mine = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float inv = __shfl_sync(0xFFFFFFFFu, inv_mine, j * 8);
    const int lost = __shfl_sync(0xFFFFFFFFu, gone, j * 8);
    if (j >= live) break;
    const int row = it.rt * R + r0 + j;
    T* out = static_cast<T*>(a.out) +
             ((it.first + row / group) * a.q_heads + it.h * group + row % group) * (int64_t)D + lane * PER;
#pragma unroll
    for (int k = 0; k < PER; k += 2)
      *reinterpret_cast<uint32_t*>(out + k) = lost ? 0u : pack2(acc[j][k] * inv, acc[j][k + 1] * inv, T());
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
template <typename T, int R, int D>
int launch_join(const AttendArgs& a, int G, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)G, R / 16);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<T, R, D>, a, G) == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
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
