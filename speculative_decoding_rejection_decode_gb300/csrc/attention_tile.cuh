// attend_tile_kernel: attention with many rows per request on the tensor cores
// (tcgen05, accumulators and weights in tensor memory).  Contracts in
// include/specdec.h (specdec_tree_attention; CROSS: specdec_cross_attention, whose keys
// are a request's filled slots alone, where its mask lets them).
//
// A unit is 128 rows x 128 keys.  Per SM one CTA:
//   loaders (2 warps)    look up the pages and bring the rows of keys and values, every
//                        second tile each, so that one's look-ups hide behind the other's,
//                        into the operand layout (swizzled rows of 128 bytes): by
//                        TMA boxes of 8 to 128 rows of a page, or by 16-byte copies
//                        where pages have odd sizes;
//   finishers (4 warps)  take a tile of values when it has landed: 8-bit ones are
//                        widened to f16 (the keys are multiplied as they are, see
//                        below); in tiles that hold nodes or miss keys, what no row
//                        may see is taken out;
//   products (1 warp)    S_w = Q K^T (both operands in shared memory), O_w += P_w V (P in
//                        tensor memory);
//   softmax (2 groups    group w takes every second tile of a segment with a
//   of 4 warps)          maximum, sum and O_w of its own, one row per thread, so
//                        that one group's exponentials overlap the other's
//                        products and nothing of a row crosses threads.
// Tensor memory: S_0, S_1 (P_w lies over S_w), O_0, O_1: 4 x 128 columns.
// The two groups' results are joined when a segment ends.
//
// Measured (32 or 64 query and 8 kv heads of 128): bf16, 2 to 9 nodes over up to 8191
// keys, 64 requests, 1.30 GB in 205 us = 6.3 TB/s; 8 nodes over 100k and 131k keys 947
// MB in 156 us = 6.1 TB/s: bound by memory.  e4m3, 29 nodes over 6000 to 16000 keys, 32
// requests: 805 MB and 177 GFLOP in 253 us, bound by the chain of roles that a tile
// passes (its scores, exponentials, weights and values widened: no unit above 41 % of
// its rate over 29 rows and 6000 states each, the softmax's and finishers' instructions
// the largest part).
//
// 8-bit keys meet the queries in e4m3 products: a query is the sum of two (f16:
// three) e4m3 parts of 4 bits each, q = hi + lo (+ lo2), which hold bf16's 8 (f16's
// 11) bits exactly down to 2^-9 (2^-6) of the row's largest value and to 2^-17 of it
// below.  That keeps the keys as they lie in memory (widening keys as well as
// values took 1.8 times as long: 32 requests of 29 nodes, 6000 to 16000 keys).  The keys' scales are applied to the scores.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention_tc.cuh"

namespace specdec {
namespace {

constexpr int kGroupWarps = 4;                       // softmax warps of a group
constexpr int kSoftmaxThreads = 2 * kGroupWarps * 32;
constexpr int kFinishWarps = 4;
constexpr int kProductWarp = 2 * kGroupWarps + kFinishWarps, kLoadWarp = kProductWarp + 2;   // (one between is idle)
constexpr int kLoaders = 2;                          // loader l takes tiles l, l + 2, ... of the range
constexpr int kTileThreads = (kProductWarp + 4) * 32;    // a whole warpgroup: registers move between those
constexpr int kW = 32;                               // scores of a row that a thread holds at once (64 took 4 % longer)
constexpr float kLeastScale = 8.673617379884035e-19f;   // 2^-60: smaller scales of values count as this
constexpr int kFactSlots = 8;                        // tiles whose key facts are held (5 are needed)

template <typename T, bool FP8, int D>
struct TileLayout {
  static constexpr int PARTS = FP8 ? (std::is_same<T, __half>::value ? 3 : 2) : 1;   // of a query
  static constexpr int QB = kR * D * (FP8 ? PARTS : 2);
  static constexpr int KB = kTK * D * (FP8 ? 1 : 2);   // a tile of keys
  static constexpr int VB = kTK * D * 2;               // a tile of values as the product takes them
  static constexpr int RB = FP8 ? kTK * D : 0;         // a tile of 8-bit values
  static constexpr int KS = FP8 && PARTS == 2 ? 4 : 3; // tiles of each in flight
  static constexpr int VS = FP8 ? 2 : 3;
  static constexpr int RS = 3;                         // landed and not yet finished (16-bit: in place)
  static constexpr int Q = 0;
  static constexpr int K = Q + QB;
  static constexpr int V = K + KS * KB;
  static constexpr int RAW = V + VS * VB;
  static constexpr int KF = RAW + (FP8 ? RS * RB : 0);             // [slot][key] scale of the key
  // [slot][key] factor of the values (f16 pair); kWide tiles: log2 of their scale
  static constexpr int VF = KF + (FP8 ? kFactSlots * kTK * 4 : 0);
  // f16 rows over 8-bit caches: values are widened exactly (by a power of two) and
  // the rest of their scale, in [1, 2), is applied to the weights in 32 bits; a
  // rounded factor and product would add two errors of f16's own size to the result
  static constexpr bool EXACT = FP8 && std::is_same<T, __half>::value;
  static constexpr int MF = VF + (FP8 ? kFactSlots * kTK * 4 : 0);   // [slot][key] that rest
  static constexpr int STATS = Q;                      // over the queries, once a segment's products are done
  static constexpr int BYTES = MF + (EXACT ? kFactSlots * kTK * 4 : 0) + 1024;   // and room to align
};

// What a tile's keys ask for besides the products.
constexpr int kClean = 0, kDirty = 1;
constexpr int kWide = 2;   // dirty, and the scales of its values differ too much for one factor

struct TileShared {
  uint64_t k_full[4], k_empty[4];
  uint64_t v_full[3], v_empty[3];
  uint64_t raw_full[3], raw_empty[3];
  uint64_t fact[kFactSlots];
  uint64_t s_full[2], p_full[2];
  uint64_t q_full, o_full;
  uint32_t live[kFactSlots][4];     // keys of a tile that the cache holds
  float vexp[kFactSlots][4];        // 8-bit caches: 32 keys' values are held as v 2^-vexp
  int dirty[kFactSlots];            // kDirty: the tile holds nodes, or misses keys; kWide as well
  float rowf[kR];
  uint32_t tmem;
  int poison;                       // some tile with nodes held a value that is not finite (stays set)
  int dead;                         // a wait ran out
};

// 8 f16 values times a pair of equal factors.
__device__ __forceinline__ uint4 times(uint4 w, uint32_t by) {
  __half2* h = reinterpret_cast<__half2*>(&w);
  const __half2 f = *reinterpret_cast<const __half2*>(&by);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __hmul2(h[i], f);
  return w;
}

// Two 16-bit weights times 2^x (a power of two, exact where it does not underflow).
__device__ __forceinline__ uint32_t shrink(uint32_t w, float by, __half) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(by));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t shrink(uint32_t w, float by, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(by));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Takes the non-finite 16-bit values out of w; whether there were any.  A row's
// hidden nodes have weight 0, and 0 x inf would reach it through the product:
// nodes' values of that kind are left out, and the rows that do see their keys get
// them when the segment ends.
template <typename E>
__device__ __forceinline__ bool clear_nonfinite(uint4& w) {
  constexpr uint32_t X = std::is_same<E, __half>::value ? 0x7C00u : 0x7F80u;
  uint32_t* u = reinterpret_cast<uint32_t*>(&w);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((u[i] & X) == X) {
      u[i] &= 0xFFFF0000u;
      any = true;
    }
    if (((u[i] >> 16) & X) == X) {
      u[i] &= 0x0000FFFFu;
      any = true;
    }
  }
  return any;
}

// Keys of tile t that a node's rows see, 128 bits; false for a malformed tree.
__device__ __forceinline__ bool visible(const Segments& s, const int32_t* all_parents, int node, int t, uint32_t* bits) {
  const int32_t* parent = all_parents ? all_parents + s.q.first : nullptr;
  const int64_t j0 = (int64_t)t * kTK - s.q.len;        // node index of the tile's first key
  // context: keys below -j0; a chain also sees the nodes up to its own
  const int64_t upto = j0 < 0 ? -j0 : 0;
  const int64_t lim = parent ? upto : max(upto, (int64_t)node + 1 - j0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t k = lim - 32 * i;
    bits[i] = k <= 0 ? 0u : (k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u);
  }
  if (!parent) return true;
  for (int x = node; x >= j0;) {
    const int64_t k = x - j0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k >= 32 * i && k < 32 * i + 32) bits[i] |= 1u << (k & 31);
    if (x == 0) break;
    const int up = __ldg(parent + x);
    if (up < 0 || up >= x) return false;
    x = up;
  }
  return true;
}

// What was left out of tiles t0 .. t1 - 1 (clear_nonfinite) for the rows of `node`:
// the values of columns d0 .. d0 + D / 2 - 1 that are not finite are added to out (or,
// where that is null, to sums).
template <typename T, bool FP8, int D>
__device__ __noinline__ void left_out(const CacheArgs& c, const Segments& s, int node, int d0, T* out, float* sums) {
  const Request& q = s.q;
  for (int t = max(s.t0, q.len / kTK); t < s.t1; ++t) {
    uint32_t bits[4];
    visible(s, c.parent, node, t, bits);
    for (int k = max(0, q.len - t * kTK); k < kTK; ++k) {   // nodes
      const int64_t at = (int64_t)t * kTK + k;
      if (at >= (int64_t)q.len + q.n) break;
      const uint32_t of = k < 32 ? bits[0] : k < 64 ? bits[1] : k < 96 ? bits[2] : bits[3];
      if (!((of >> (k & 31)) & 1u)) continue;
      const int64_t r0 = cache_row(c.geo, c.table + s.b * c.geo.table_stride, at);
      if (r0 < 0) continue;
      const int64_t r = r0 + (int64_t)s.h * c.geo.page_size;
#pragma unroll 4
      for (int d = d0; d < d0 + D / 2; ++d) {
        float v;
        if constexpr (FP8) {
          const __half_raw e = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(c.v)[r * D + d], __NV_E4M3);
          v = __half2float(*reinterpret_cast<const __half*>(&e)) * c.vs[r];
        } else {
          v = to_float(static_cast<const T*>(c.v)[r * D + d]);
        }
        if (isfinite(v)) continue;
        if (out) from_float(to_float(out[d]) + v, out[d]);
        else sums[d] += v;
      }
    }
  }
}

// One tile's scores of this thread's row become weights: one pass, kW keys at a time.
// Weights are 2^(e - m), m the first maximum (so that a row that sees one key gets its
// values as they are), which follows the running maximum by whole numbers and only when
// that is kLazy above it: what has been summed, the row's O_w (`summed`: there is
// one) and the tile's weights so far are then multiplied by 2^(m - m').  m' = m + k is rounded to
// 32 bits, so that the factor is a power of two but for |m'| 2^-24, as much as the scores of
// that size are off by themselves; the weights' own factor is rounded to their 16 bits, to
// the power of two.  The largest weight lies in [2^kHead, 2^(kHead + kLazy)]: f16 weights keep
// their bits far below the largest, and the maximum may lag by 2^kLazy.
template <typename T, bool FP8, int D, bool WIDE>
__device__ __forceinline__ void tile_scores(uint32_t ts, uint32_t to, uint32_t base_s, int f, const float* vexp,
                                            const uint32_t* bits, bool masked, float rowf, bool summed, float& m, float& l) {
  using L = TileLayout<T, FP8, D>;
  using E = typename std::conditional<FP8, __half, T>::type;
  // f16 ends at 2^16: a weight of at most 2^15, or of 2^14 where it is yet to be multiplied with
  // the rest of a scale (EXACT, below 2).  8-bit caches, 8 and 9: 180 and 175 us, 32 requests of
  // 29 bf16 rows over 1500 to 12000 states; bf16 weights, 9 and 16: 208 and 205, 64 of 2 to 9
  // over up to 8191 keys.  bf16 weights end at 1, so that sums pass no further than the sum of
  // the values' magnitudes.
  constexpr float kLazy = L::EXACT ? 8.0f : std::is_same<E, __half>::value ? 9.0f : 16.0f;
  constexpr float kHead = std::is_same<E, __half>::value ? 6.0f : -kLazy;
#pragma unroll 1
  for (int i = 0; i < kTK / kW; ++i) {
    const float of = WIDE ? 1.0f : rowf;   // kWide: in the scores already
    const uint64_t rowf2 = pair(of, of);
    float s[kW], shift = 0.0f;
    if constexpr (FP8 && !WIDE) shift = vexp[i];   // 8-bit caches: the values' exponent
    tc_ld32(ts + i * kW, s);
    if constexpr (FP8) {
#pragma unroll
      for (int k = 0; k < kW; k += 16) {
        uint64_t kf[8];
        lds_pairs(base_s + L::KF + (f * kTK + i * kW + k) * 4, kf);
#pragma unroll
        for (int z = 0; z < 8; ++z) unpair(mul2(pair(s[k + 2 * z], s[k + 2 * z + 1]), kf[z]), s[k + 2 * z], s[k + 2 * z + 1]);
      }
    }
    if (masked) {
      const uint32_t see = i == 0 ? bits[0] : i == 1 ? bits[1] : i == 2 ? bits[2] : bits[3];
      if constexpr (WIDE) {
        const uint64_t row2 = pair(rowf, rowf);
#pragma unroll
        for (int k = 0; k < kW; k += 16) {
          uint64_t lv[8];
          lds_pairs(base_s + L::VF + (f * kTK + i * kW + k) * 4, lv);
#pragma unroll
          for (int z = 0; z < 8; ++z)
            unpair(fma2(pair(s[k + 2 * z], s[k + 2 * z + 1]), row2, lv[z]), s[k + 2 * z], s[k + 2 * z + 1]);
        }
      }
#pragma unroll
      for (int k = 0; k < kW; ++k)
        if (!((see >> k) & 1u)) s[k] = -INFINITY;
    }
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = fmaxf(s[2 * k], s[2 * k + 1]);
#pragma unroll
    for (int k = 8; k < kW; k += 8)
#pragma unroll
      for (int x = 0; x < 4; ++x) q[x] = max3(q[x], s[k + 2 * x], s[k + 2 * x + 1]);
    const float mx = fmaxf(max3(q[0], q[1], q[2]), q[3]);
    const float most = mx == -INFINITY ? mx : fmaf(mx, of, shift);
    const bool move = most > m + kLazy || (m == -INFINITY && most != -INFINITY);
    if (__any_sync(0xFFFFFFFFu, move)) {
      const float to_m = !move ? m : m == -INFINITY ? most : m + ceilf(most - m);
      const float fix = move ? ex2(m - to_m) : 1.0f;
      m = to_m;
      if (summed || i > 0) {
        tc_wait_st();   // what is read back here has been stored
        l *= fix;
        if (i > 0) {
#pragma unroll 1
          for (int p = 0; p < i; ++p) {
            uint32_t w16[16];
            tc_ld16(ts + p * 16, w16);
#pragma unroll
            for (int k = 0; k < 16; ++k) w16[k] = shrink(w16[k], fix, E());
            tc_st16(ts + p * 16, w16);
          }
        }
        if (summed) {
#pragma unroll 1
          for (int p = 0; p < D / 16; ++p) {
            uint32_t o[16];
            tc_ld16(to + p * 16, o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fix);
            tc_st16(to + p * 16, o);
          }
        }
      }
    }
    // weights, rounded to 16 bits for the product with V (half a step
    // each at most) and summed unrounded
    const float ref = (m == -INFINITY ? 0.0f : m) - kHead;
    const float add = shift - ref;
    const uint64_t add_2 = pair(add, add);
    uint64_t sum[2] = {0, 0};
    if constexpr (WIDE) {   // exponentials of their own: the weights may underflow where these do not
#pragma unroll
      for (int k = 0; k < kW; k += 16) {
        uint64_t lv[8];
        lds_pairs(base_s + L::VF + (f * kTK + i * kW + k) * 4, lv);
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          const float s0 = s[k + 2 * z], s1 = s[k + 2 * z + 1];
          float a0, a1;
          unpair(lv[z], a0, a1);
          sum[z & 1] = add2(sum[z & 1], pair(s0 == -INFINITY ? 0.0f : ex2(s0 + add - a0), s1 == -INFINITY ? 0.0f : ex2(s1 + add - a1)));
        }
      }
    }
    uint32_t p[kW / 2];
    constexpr bool REST = L::EXACT && !WIDE;
    [[maybe_unused]] uint64_t rest[REST ? kW / 2 : 1];   // of the values' scales
    if constexpr (REST) {
      lds_pairs(base_s + L::MF + (f * kTK + i * kW) * 4, rest);
      lds_pairs(base_s + L::MF + (f * kTK + i * kW) * 4 + 64, rest + 8);
    }
#pragma unroll
    for (int k = 0; k < kW; k += 2) {
      float e0, e1;
      unpair(fma2(pair(s[k], s[k + 1]), rowf2, add_2), e0, e1);
      e0 = ex2(e0);
      e1 = ex2(e1);
      if constexpr (!WIDE) sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pair(e0, e1));
      if constexpr (REST) unpair(mul2(pair(e0, e1), rest[k / 2]), e0, e1);
      p[k / 2] = pack2(e0, e1, E());
    }
    tc_st16(ts + i * (kW / 2), p);
    float s0, s1;
    unpair(add2(sum[0], sum[1]), s0, s1);
    if constexpr (FP8) l = fmaf(s0 + s1, WIDE ? 1.0f : __uint_as_float((uint32_t)(127 - (int)shift) << 23), l);
    else l += s0 + s1;
  }
}

// The same for kWide tiles, out of line: they are rare, and their code among the
// others' cost all tiles 4 to 8 % (299 us -> 312 to 325).
template <typename T, bool FP8, int D>
__device__ __noinline__ float2 wide_scores(uint32_t ts, uint32_t to, uint32_t base_s, int f, uint4 see, float rowf,
                                           bool summed, float m, float l) {
  const uint32_t bits[4] = {see.x, see.y, see.z, see.w};
  tile_scores<T, FP8, D, true>(ts, to, base_s, f, nullptr, bits, true, rowf, summed, m, l);
  return make_float2(m, l);
}

// Whether a tile with nodes is a kWide one, by the scales of its values (4 a lane;
// `most`: the largest of 32 keys, as bits); what the other roles need is then written
// here, out of line for the same reason.
template <typename T, int D>
__device__ __noinline__ bool wide_facts(char* smem, int f, float4 vs, uint32_t most) {
  using L = TileLayout<T, true, D>;
  const int lane = threadIdx.x & 31;
  const float* vv = &vs.x;
  uint32_t least = most;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (vv[k] > 0.0f) least = min(least, __float_as_uint(vv[k]));
  if (!__any_sync(0xFFFFFFFFu, (most >> 23) > (least >> 23) + 20)) return false;
  float lv[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) lv[k] = vv[k] == vv[k] ? __log2f(fmaxf(vv[k], kLeastScale)) : vv[k];
  reinterpret_cast<float4*>(smem + L::VF)[f * (kTK / 4) + lane] = make_float4(lv[0], lv[1], lv[2], lv[3]);
  return true;
}

template <typename T, bool FP8, int D, bool CROSS>
__global__ void __launch_bounds__(kTileThreads, 1)
    attend_tile_kernel(const AttendArgs a, const int box, const bool grouped, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using L = TileLayout<T, FP8, D>;
  using E = typename std::conditional<FP8, __half, T>::type;
  constexpr int CH = D / 8;                      // 16-byte chunks of an operand row
  extern __shared__ char smem_raw[];
  __shared__ ScanShared scan;
  __shared__ __align__(8) TileShared sh;
  // segments of the softmax groups, the products, the loaders and the finishers
  __shared__ Segments segs[3 + kLoaders];
  char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base_s = smem_addr(smem);
  const CacheArgs& c = a.c;
  const int G = gridDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.q_heads / c.geo.kv_heads;
  const PlanArgs plan(a);
  uint32_t why = 0;
  int64_t u0 = 0;
  find_unit<kTileThreads>(plan, kR, kTK,
                          [&](int64_t units) {
                            const int ranges = (int)min((int64_t)G, units);
                            u0 = (int)blockIdx.x < ranges ? range_begin(units, ranges, blockIdx.x) : units;
                            return u0;
                          },
                          scan, why);
  if (blockIdx.x == 0 && why) atomicOr(c.err, why);
  if (tid == 0 && !a.whole) Partials<kR, D>(a.workspace, G).open[blockIdx.x].ranges = 0;
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t units = scan.total;
  const int ranges = (int)min((int64_t)G, units);
  if ((int)blockIdx.x >= ranges || scan.b < 0) return;
  if (tid == 0) {
    for (int i = 0; i < L::KS; ++i) {
      mbar_init(smem_addr(&sh.k_full[i]), 32);
      mbar_init(smem_addr(&sh.k_empty[i]), 1);
    }
    for (int i = 0; i < L::VS; ++i) {
      mbar_init(smem_addr(&sh.v_full[i]), kFinishWarps * 32);
      mbar_init(smem_addr(&sh.v_empty[i]), 1);
    }
    for (int i = 0; i < L::RS; ++i) {
      mbar_init(smem_addr(&sh.raw_full[i]), 32);
      mbar_init(smem_addr(&sh.raw_empty[i]), kFinishWarps);
    }
    for (int i = 0; i < kFactSlots; ++i) mbar_init(smem_addr(&sh.fact[i]), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_addr(&sh.s_full[w]), 1);
      mbar_init(smem_addr(&sh.p_full[w]), kGroupWarps);
    }
    mbar_init(smem_addr(&sh.q_full), 2 * kGroupWarps);
    mbar_init(smem_addr(&sh.o_full), 2);   // the products' end, and the thread that issued them
    sh.poison = 0;
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == kProductWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "n"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sh.tmem;
  const int64_t uend = range_begin(units, ranges, blockIdx.x + 1);
  if (tid < 3 + kLoaders) {
    uint32_t ignored = 0;
    Segments& s = segs[tid];
    s.end = uend;
    s.b = scan.b;
    s.base = scan.before;
    s.u = (int)(u0 - scan.before);
    s.q = attend_request(plan, scan.b, kR, kTK, ignored);
    next_segment<kR>(&s, plan);
  }
  __syncthreads();
  uint32_t bad = 0;

  // Registers: 4 warpgroups are launched with 128 a thread.  The softmax groups take
  // 40 more each from the two others (168 + 168 + 72 + 104 = 4 * 128).
  auto wait_use = [&](uint64_t* bars, int slots, int n) {       // use n of a ring's slot is complete
    wait_or_give_up(sh.dead, smem_addr(&bars[n % slots]), (uint32_t)(n / slots) & 1u);
  };
  auto wait_free = [&](uint64_t* bars, int slots, int n) {      // the slot's use n - slots is complete
    wait_or_give_up(sh.dead, smem_addr(&bars[n % slots]), ((uint32_t)(n / slots) & 1u) ^ 1u);
  };
  if (warp >= kProductWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kProductWarp) {
      // ---- products ---------------------------------------------------------------
      // One warp for all of them, in the order ... P_w V of a tile, S_w of the tile after next
      // ...: the tensor cores take products up in order, so that S_w may follow P_w V at once
      // although it lies over P_w (with a warp each for scores and weighted values, scores
      // waited for the other's products to end and be seen).
      Segments& seg = segs[1];
      const uint32_t tmu = __shfl_sync(0xFFFFFFFFu, tm, 0), ops = __shfl_sync(0xFFFFFFFFu, base_s, 0);
      auto scores = [&](int w, int n) {            // of tile n; the elected thread's
        const uint32_t kt = ops + L::K + (n % L::KS) * L::KB;
        if constexpr (FP8) {
          const uint64_t kd = operand<D>(kt, 16);
#pragma unroll
          for (int part = 0; part < L::PARTS; ++part) {
            const uint64_t qd = operand<D>(ops + L::Q + part * kR * D, 16);
#pragma unroll
            for (int s = 0; s < D / 32; ++s)
              tc_mma_e4m3(tmu + w * 128, qd + s * 2, kd + s * 2, product_e4m3(kTK), part + s > 0);
          }
        } else {
          const uint64_t qd = operand(ops + L::Q, 16), kd = operand(kt, 16);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = (uint32_t)((s >> 2) * (kTK * 128) + (s & 3) * 32) >> 4;
            tc_mma_ss(tmu + w * 128, qd + off, kd + off, product<E>(kTK, false), s > 0);
          }
        }
        tc_commit(smem_addr(&sh.s_full[w]));
        tc_commit(smem_addr(&sh.k_empty[n % L::KS]));
      };
      auto keys = [&](int n) {
        wait_use(sh.k_full, L::KS, n);
        fence_async_proxy();   // rows that came by 16-byte copies
        tc_fence_after();
      };
      int k = 0;                                  // tiles so far
      uint32_t used = 0;                          // bit w: phase of group w's weights
      for (uint32_t g = 0; seg.more; ++g) {
        const int n = seg.t1 - seg.t0;
        wait_or_give_up(sh.dead, smem_addr(&sh.q_full), g & 1u);
#pragma unroll 1
        for (int j = 0; j < 2 && j < n; ++j) {
          keys(k + j);
          if (tc_elect()) scores(j, k + j);
          __syncwarp();
        }
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++k) {
          const int w = j & 1;
          wait_use(sh.v_full, L::VS, k);
          if (j + 2 < n) keys(k + 2);
          wait_or_give_up(sh.dead, smem_addr(&sh.p_full[w]), (used >> w) & 1u);
          used ^= 1u << w;
          tc_fence_after();
          if (tc_elect()) {
            const uint64_t vd = operand(ops + L::V + (k % L::VS) * L::VB, kTK * 128);
#pragma unroll
            for (int s = 0; s < kTK / 16; ++s)
              tc_mma_ts(tmu + 256 + w * 128, tmu + w * 128 + s * 8, vd + (uint32_t)(s * 2048 >> 4), product<E>(D, true),
                        s > 0 || j >= 2);
            tc_commit(smem_addr(&sh.v_empty[k % L::VS]));
            if (j + 2 < n) scores(w, k + 2);
            if (j + 1 == n) tc_commit(smem_addr(&sh.o_full));
          }
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive(smem_addr(&sh.o_full));
          next_segment<kR>(&seg, plan);
        }
        __syncwarp();
      }
    } else if (warp >= kLoadWarp) {
      // ---- loaders ----------------------------------------------------------------
      // Pages that are a multiple of 32 slots (`grouped`): 32 keys from a multiple of
      // 32 lie in one page, so lanes 0 .. 3 look up one page each and hold the cache
      // row and the live keys of their 32; else a lane looks after keys lane, lane +
      // 32, ...  (The common way is kept short: straight code that runs once a tile
      // comes from beyond the instruction cache each time.)
      const int loader = warp - kLoadWarp;
      const uint32_t one = lane == 0 ? 1u : 0u;
      const uint32_t page_size = (uint32_t)c.geo.page_size;
      struct Place {
        const int32_t* pages;
        uint32_t first, len, end;
        int h, id;
        uint32_t see;                           // masks: bit i is key 32 i + lane's
      };
      Segments& seg = segs[2 + loader];
      int skip = loader, t = seg.t0;            // tiles of others before this loader's next
      // The next item's queries on their way to L2 while this one's last tiles are worked on:
      // 32 requests of 29 rows over 1500 to 12000 8-bit states 184 to 178 us, 64 of 2 to 9 over
      // up to 8191 195 to 179 (but the 8-bit attention over context and nodes 255 to 271, whose
      // roles' code is the longest: it goes without).
      auto fetch_queries = [&](const Segments& s) {
#pragma unroll 1
        for (int i = lane; i < s.rows * (D / 64); i += 32) {
          const int gr = s.rt * kR + i / (D / 64);
          const T* src = static_cast<const T*>(a.q) + (s.q.first + gr / group) * a.q_row + (int64_t)(s.h * group + gr % group) * a.q_head + i % (D / 64) * 64;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
        }
      };
      auto go = [&](Place& x) -> bool {         // this loader's next tile
        t += skip;
        while (seg.more && t >= seg.t1) {
          const int over = t - seg.t1;
          __syncwarp();
          if (lane == 0) next_segment<kR>(&seg, plan);
          __syncwarp();
          t = seg.t0 + over;
          if ((CROSS || !FP8) && loader == 0 && seg.more) fetch_queries(seg);
        }
        if (!seg.more) return false;
        skip = kLoaders;
        x.pages = c.table + seg.b * c.geo.table_stride;
        x.len = (uint32_t)seg.q.len;
        x.end = CROSS ? x.len : x.len + (uint32_t)seg.q.n;      // within the table
        x.first = (uint32_t)t * kTK;
        x.h = seg.h;
        x.id = -1;
        const uint32_t at = x.first + lane * 32;
        if (grouped && lane < 4 && at < x.end) x.id = __ldg(x.pages + at / page_size);
        if constexpr (CROSS) {
          x.see = 15u;
          if (a.mask) {
            x.see = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int64_t s = (int64_t)x.first + i * 32 + lane;
              if (s < x.end && s < a.mask_slots && __ldg(a.mask + seg.b * a.mask_stride + s)) x.see |= 1u << i;
            }
          }
        }
        return true;
      };
      // fewer than 2^31 rows in all; -1: the cache does not hold the slot
      auto row_at = [&](const Place& x, int id, uint32_t at) -> int {
        return id >= 0 && id < c.geo.num_pages ? (id * c.geo.kv_heads + x.h) * (int)page_size + (int)(at % page_size) : -1;
      };
      // The rows of a tile of the array `src` (16-bit, or 8-bit as it is) to `dst`;
      // every lane arrives on `bar` when its copies have landed.  A box lies within
      // one page: it is fetched if its first key lives, and what it brings of slots
      // behind the last key is hidden (keys) or taken out (values).
      constexpr int LINE = FP8 ? D : 128, HALVES = FP8 ? 1 : D / 64, RC = FP8 ? D / 16 : D / 8;
      auto load_box = [&](uint32_t dst, const CUtensorMap* map, int r0, int row, uint32_t bar) {
#pragma unroll
        for (int half = 0; half < HALVES; ++half)
          box_load(dst + half * (kTK * 128) + r0 * LINE, map, half * 64, row, bar, one);
      };
      auto fetch_grouped = [&](uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
        const unsigned firsts = __ballot_sync(0xFFFFFFFFu, lane < 4 && (lane * 32) % box == 0 && row >= 0);
        if (one) mbar_expect_tx(bar, __popc(firsts) * box * HALVES * LINE);
        // a lane for each box
        const int i = lane / HALVES, half = lane % HALVES, r = __shfl_sync(0xFFFFFFFFu, row, i);
        if (i < 4 && ((firsts >> i) & 1u)) box_load(dst + half * (kTK * 128) + i * 32 * LINE, map, half * 64, r, bar, 1u);
        mbar_arrive(bar);
      };
      auto fetch_any = [&](uint32_t dst, const void* src, const CUtensorMap* map, const int* row, uint32_t bar) {
        const uint32_t firsts = box == 16 ? 0x00010001u : 0x01010101u;   // first keys of boxes among 32
        int count = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) count += __popc(__ballot_sync(0xFFFFFFFFu, row[i] >= 0) & firsts);
        if (one && box > 0) mbar_expect_tx(bar, count * box * HALVES * LINE);
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int mine = i == 0 ? row[0] : i == 1 ? row[1] : i == 2 ? row[2] : row[3];
          if (box > 0) {
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += box) {
              const int r = __shfl_sync(0xFFFFFFFFu, mine, r0);
              if (r >= 0) load_box(dst, map, i * 32 + r0, r, bar);
            }
          } else {
#pragma unroll 4
            for (int z = 0; z < RC; ++z) {
              const int y = z * 32 + lane, key = y / RC, ch = y % RC;
              const int r = __shfl_sync(0xFFFFFFFFu, mine, key);
              copy16(dst + (FP8 ? byte_chunk<D>(i * 32 + key, ch) : op_chunk(i * 32 + key, ch)),
                     static_cast<const char*>(src) + (int64_t)max(r, 0) * (FP8 ? D : 2 * D) + ch * 16, r >= 0);
            }
          }
        }
        copy_arrive(bar);
      };
      Place ahead;
      bool have = go(ahead);
      for (int n = loader; have; n += kLoaders) {
        const Place now = ahead;
        const bool tail = now.first + kTK > now.len;
        int row = -1, rows[4] = {-1, -1, -1, -1};
        uint32_t live = 0, missed = 0;           // lanes 0 .. 3: of their 32 keys; grouped: those without a page
        if (grouped) {
          const uint32_t at = now.first + lane * 32;
          if (lane < 4 && at < now.end) {
            row = row_at(now, now.id, at);
            (row >= 0 ? live : missed) = now.end - at >= 32 ? 0xFFFFFFFFu : (1u << (now.end - at)) - 1u;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t at = now.first + i * 32 + lane;
            rows[i] = row_at(now, at < now.end ? __ldg(now.pages + at / page_size) : -1, at);
            const uint32_t l = __ballot_sync(0xFFFFFFFFu, rows[i] >= 0);
            if (lane == i) live = l;
            if (at < now.end && rows[i] < 0 && (!CROSS || ((now.see >> i) & 1u))) bad |= SPECDEC_DEVERR_BAD_CACHE;
          }
        }
        if constexpr (CROSS) {
          if (a.mask) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t l = __ballot_sync(0xFFFFFFFFu, (now.see >> i) & 1u);
              if (lane == i) {
                live &= l;
                missed &= l;                     // a masked slot needs no page
              }
            }
          }
        }
        if (missed) bad |= SPECDEC_DEVERR_BAD_CACHE;
        const bool dirty = tail || __any_sync(0xFFFFFFFFu, lane < 4 && live != 0xFFFFFFFFu);
        // scales, 4 neighbouring keys a lane
        float4 ks = make_float4(0.0f, 0.0f, 0.0f, 0.0f), vs = ks;
        uint32_t seen = 0;                       // which of the 4 live
        if constexpr (FP8) {
          const int sub = (lane & 7) * 4;
          seen = __shfl_sync(0xFFFFFFFFu, live, lane >> 3) >> sub;
          if (grouped) {
            const int r = __shfl_sync(0xFFFFFFFFu, row, lane >> 3);
            if (r >= 0) {
              ks = __ldg(reinterpret_cast<const float4*>(c.ks + r + sub));
              vs = __ldg(reinterpret_cast<const float4*>(c.vs + r + sub));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              int r = -1;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int x = __shfl_sync(0xFFFFFFFFu, rows[i], sub + k);
                if ((lane >> 3) == i) r = x;
              }
              (&ks.x)[k] = r >= 0 ? __ldg(c.ks + r) : 0.0f;
              (&vs.x)[k] = r >= 0 ? __ldg(c.vs + r) : 0.0f;
            }
          }
        }
        have = go(ahead);
        const uint32_t kdst = base_s + L::K + (n % L::KS) * L::KB, kbar = smem_addr(&sh.k_full[n % L::KS]);
        const uint32_t vdst = base_s + (FP8 ? L::RAW + (n % L::RS) * L::RB : L::V + (n % L::VS) * L::VB);
        const uint32_t vbar = smem_addr(&sh.raw_full[n % L::RS]);
        wait_free(sh.k_empty, L::KS, n);
        if (grouped) fetch_grouped(kdst, &kmap, row, kbar);
        else fetch_any(kdst, c.k, &kmap, rows, kbar);
        wait_free(sh.raw_empty, L::RS, n);
        if constexpr (!FP8) wait_free(sh.v_empty, L::VS, n);   // landing in place
        if (grouped) fetch_grouped(vdst, &vmap, row, vbar);
        else fetch_any(vdst, c.v, &vmap, rows, vbar);
        // What the other roles need to know of the tile's keys.  8-bit caches: the
        // scale of K (applied to the scores, in 32 bits); the scale of V goes into
        // the widened values, as a factor v 2^-vexp that f16 holds: the largest of
        // 32 keys lies in [2^5, 2^6), so products stay below 2^15 and keys down to
        // 2^-20 of the largest keep f16's full precision (bf16 rows: the factor and
        // its products with the values are rounded to f16, an eighth of what the
        // result's own rounding is).
        // That serves keys which every row sees.  In a tile with nodes a row must not
        // lose bits to the scale of a key that is hidden from it.  Where such a tile's
        // scales are more than 2^20 apart (kWide) the values are widened as they are,
        // log2 of the scale is added to the scores, so that each row's weights carry the
        // scales of the keys that it sees; their sum is of the weights without them.
        // (All tiles with nodes that way: 64 requests of 9 nodes 281 us instead of 257.)
        // (Slot n % 8 is free: the slot waits above imply that the products of tile
        // n - 5 are done.)
        const int f = n % kFactSlots;
        if (lane < 4) sh.live[f][lane] = live;
        int kind = dirty ? kDirty : kClean;
        if constexpr (FP8) {
          float* kk = &ks.x;
          float* vv = &vs.x;
          uint32_t most = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool in = (seen >> k) & 1u;
            if (!in) kk[k] = vv[k] = 0.0f;
            if (vv[k] > 0.0f && isfinite(vv[k])) most = max(most, __float_as_uint(vv[k]));
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
          if (dirty && wide_facts<T, D>(smem, f, vs, most)) kind = kWide;
          const int b = most ? max((int)(most >> 23) - 127 - 5, -80) : 0;   // 122 at most
          const float by = __uint_as_float((uint32_t)(127 - b) << 23);
          if ((lane & 7) == 0) sh.vexp[f][lane >> 3] = (float)b;
          reinterpret_cast<float4*>(smem + L::KF)[f * (kTK / 4) + lane] = ks;
          if (kind != kWide) {
            if constexpr (L::EXACT) {
              float rest[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t e = __float_as_uint(vv[k]) & 0x7F800000u;   // 2^exponent
                const bool split = e != 0 && e != 0x7F800000u;
                rest[k] = split ? vv[k] / __uint_as_float(e) : 1.0f;       // exact
                if (split) vv[k] = __uint_as_float(e);
              }
              reinterpret_cast<float4*>(smem + L::MF)[f * (kTK / 4) + lane] = make_float4(rest[0], rest[1], rest[2], rest[3]);
            }
            reinterpret_cast<uint4*>(smem + L::VF)[f * (kTK / 4) + lane] =
                make_uint4(pack2(vv[0] * by, vv[0] * by, __half()), pack2(vv[1] * by, vv[1] * by, __half()),
                           pack2(vv[2] * by, vv[2] * by, __half()), pack2(vv[3] * by, vv[3] * by, __half()));
          }
        }
        if (lane == 0) sh.dirty[f] = kind;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.fact[f]));
      }
      copy_commit();
      copy_wait<0>();
    }
  } else if (warp >= 2 * kGroupWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---- finishers: 32 keys each.  8 lanes read and write one chunk of 8
    // neighbouring rows, without bank conflicts in any of the swizzles ------------
    const int pw = warp - 2 * kGroupWarps;
    Segments& seg = segs[2 + kLoaders];
    for (int n = 0, t = seg.t0; seg.more; ++n) {
      const int f = n % kFactSlots;
      wait_use(sh.fact, kFactSlots, n);
      const bool dirty = sh.dirty[f] != kClean;
      const uint32_t live = sh.live[f][pw];
      const int nodes = seg.q.len - t * kTK - pw * 32;      // the warp's keys from here on are nodes
      const uint32_t dst = base_s + L::V + (n % L::VS) * L::VB;
      uint32_t own = 0;
      if constexpr (FP8) {
        own = reinterpret_cast<const uint32_t*>(smem + L::VF)[f * kTK + pw * 32 + lane];
        if (sh.dirty[f] == kWide) own = 0x3C003C00u;   // 1: the scales are in the weights
      }
      wait_use(sh.raw_full, L::RS, n);
      bool hit = false;
      if constexpr (FP8) {
        wait_free(sh.v_empty, L::VS, n);
        const uint32_t raw = base_s + L::RAW + (n % L::RS) * L::RB;
        constexpr int RC = D / 16;             // 16-byte chunks of an 8-bit row
#pragma unroll 2
        for (int i = 0; i < RC; ++i) {
          const int in = (lane & 7) + 8 * (RC == 8 ? i >> 1 : i), key = pw * 32 + in;
          const int ch = (lane >> 3) + (RC == 8 ? 4 * (i & 1) : 0);
          const uint4 w = lds128(raw + byte_chunk<D>(key, ch));
          const uint32_t by = __shfl_sync(0xFFFFFFFFu, own, in);
          uint4 lo = times(make_uint4(e4m3x2_f16x2(w.x), e4m3x2_f16x2(w.x >> 16), e4m3x2_f16x2(w.y), e4m3x2_f16x2(w.y >> 16)), by);
          uint4 hi = times(make_uint4(e4m3x2_f16x2(w.z), e4m3x2_f16x2(w.z >> 16), e4m3x2_f16x2(w.w), e4m3x2_f16x2(w.w >> 16)), by);
          sts128(dst + op_chunk(key, 2 * ch), lo);
          sts128(dst + op_chunk(key, 2 * ch + 1), hi);
        }
        __syncwarp();
      }
      if (dirty && (nodes < 32 || live != 0xFFFFFFFFu)) {
#pragma unroll 1
        for (int i = 0; i < CH; ++i) {
          const int in = (lane & 7) + 8 * (i & 3), ch = (lane >> 3) + 4 * (i >> 2);
          const uint32_t at = dst + op_chunk(pw * 32 + in, ch);
          if (!((live >> in) & 1u)) {
            sts128(at, make_uint4(0, 0, 0, 0));
          } else if (in >= nodes) {
            uint4 w = lds128(at);
            if (clear_nonfinite<E>(w)) {
              sts128(at, w);
              hit = true;
            }
          }
        }
      }
      if (hit) *reinterpret_cast<volatile int*>(&sh.poison) = 1;
      fence_async_proxy();
      mbar_arrive(smem_addr(&sh.v_full[n % L::VS]));
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.raw_empty[n % L::RS]));
      if (++t == seg.t1) {
        named_bar_sync(2, kFinishWarps * 32);
        if (warp == 2 * kGroupWarps && lane == 0) next_segment<kR>(&seg, plan);
        named_bar_sync(2, kFinishWarps * 32);
        t = seg.t0;
      }
    }
  } else {
    // ---- softmax ----------------------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int w = warp / kGroupWarps;            // group: tiles w, w + 2, ... of a segment
    const int row = (warp % kGroupWarps) * 32 + lane;   // row of the tile = lane of tensor memory
    const uint32_t lanes = (uint32_t)(warp % kGroupWarps) << 21;   // first lane, in bits 16..
    const uint32_t ts = tm + lanes + w * 128, to = tm + lanes + 256 + w * 128;
    const int sid = tid;                         // 0 .. 255
    float2* stats = reinterpret_cast<float2*>(smem + L::STATS);
    const Partials<kR, D> part(a.workspace, G);
    int done = 0, tile0 = 0;                     // this group's tiles, all tiles before the segment
    uint32_t g = 0;
    // The segment stands in shared memory: its fields would otherwise take the
    // registers of the scores.
    Segments& seg = segs[0];
    while (seg.more) {
      // queries
      const float sgn = a.scale_log2 < 0.0f ? -1.0f : 1.0f;   // factors are positive: the sign goes to q
      constexpr int kAhead = FP8 ? 2 : 4;   // loads in flight
#pragma unroll kAhead
      for (int x = sid; x < kR * CH; x += kSoftmaxThreads) {
        const int r = x / CH, ch = x % CH;
        const bool live = r < seg.rows;
        const int gr = seg.rt * kR + (live ? r : 0);
        const T* src = static_cast<const T*>(a.q) + (seg.q.first + gr / group) * a.q_row +
                       (int64_t)(seg.h * group + gr % group) * a.q_head + ch * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = __ldg(reinterpret_cast<const uint4*>(src));
        float f = fabsf(a.scale_log2);
        if constexpr (FP8) {
          // the row is scaled by a power of two so that its largest value lies in
          // [2^7, 2^8), below e4m3's 448; the scores take the factor back
          const T* e = reinterpret_cast<const T*>(&v);
          float y[8], m = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            y[i] = to_float(e[i]) * sgn;
            m = fmaxf(m, fabsf(y[i]));
          }
#pragma unroll
          for (int o = CH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const int ex = min(max((int)(__float_as_uint(m) >> 23), 8), 253);
          const float mul = __uint_as_float((uint32_t)(254 - ex + 7) << 23);
          f *= __uint_as_float((uint32_t)(ex - 7) << 23);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = isfinite(y[i]) ? y[i] * mul : __uint_as_float(0x7FC00000u);
#pragma unroll
          for (int part = 0; part < L::PARTS; ++part) {
            uint32_t w8[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(y[i], y[i + 1]), __NV_SATFINITE, __NV_E4M3);
              w8[i >> 2] |= two << ((i & 2) * 8);
              const uint32_t back = e4m3x2_f16x2(two);
              const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&back));
              y[i] -= got.x;
              y[i + 1] -= got.y;
            }
            sts64(base_s + L::Q + part * kR * D + byte_chunk<D>(r, ch >> 1) + (ch & 1) * 8, w8[0], w8[1]);
          }
        } else if (sgn < 0.0f) {
          v.x ^= 0x80008000u;
          v.y ^= 0x80008000u;
          v.z ^= 0x80008000u;
          v.w ^= 0x80008000u;
        }
        if constexpr (!FP8) sts128(base_s + L::Q + op_chunk(r, ch), v);
        if (ch == 0) sh.rowf[r] = fmaxf(f, 1.17549435e-38f);   // above 0: hidden keys are -inf times this
      }
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.q_full));
      named_bar_sync(1, kSoftmaxThreads);
      const float rowf = sh.rowf[row];
      const int t0 = seg.t0, n = seg.t1 - t0, len = seg.q.len;
      const bool busy = (row & ~31) < seg.rows;    // the warp has rows of the tile
      const int node = (seg.rt * kR + min(row, seg.rows - 1)) / group;
      float m = -INFINITY, l = 0.0f;               // reference maximum and sum of this group's tiles
      bool lost = false;                           // the row's node has no walk to node 0
      for (int j = w; j < n; j += 2) {
        const int t = t0 + j, f = (tile0 + j) % kFactSlots;
        wait_use(sh.fact, kFactSlots, tile0 + j);
        wait_or_give_up(sh.dead, smem_addr(&sh.s_full[w]), (uint32_t)done & 1u);
        ++done;
        tc_fence_after();
        if (busy) {
          uint32_t bits[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
          const bool tail = (int64_t)t * kTK + kTK > len;
          if (!CROSS && tail && !visible(seg, c.parent, node, t, bits)) lost = true;
          __syncwarp();
          bool masked = tail;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t lv = sh.live[f][i];
            masked |= lv != 0xFFFFFFFFu;
            bits[i] &= lv;
          }
          if (FP8 && masked && sh.dirty[f] == kWide) {
            const float2 ml = wide_scores<T, FP8, D>(ts, to, base_s, f, make_uint4(bits[0], bits[1], bits[2], bits[3]), rowf, j >= 2, m, l);
            m = ml.x;
            l = ml.y;
          } else {
            tile_scores<T, FP8, D, false>(ts, to, base_s, f, sh.vexp[f], bits, masked, rowf, j >= 2, m, l);
          }
          tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[w]));
      }
      // ---- the segment's end: both groups' results joined, half of the head each
      wait_or_give_up(sh.dead, smem_addr(&sh.o_full), g & 1u);
      tc_fence_after();
      if (lost) bad |= SPECDEC_DEVERR_BAD_TREE;
      stats[w * kR + row] = make_float2(m, lost ? kLostRow : l);
      named_bar_sync(1, kSoftmaxThreads);
      if (busy) {
        float2 s0 = stats[row], s1 = stats[kR + row];
        const bool gone = s0.y == kLostRow || s1.y == kLostRow;
        if (gone) s0 = s1 = make_float2(-INFINITY, 0.0f);   // a row of zeros
        const float mm = fmaxf(s0.x, s1.x), ref = mm == -INFINITY ? 0.0f : mm;
        const float f0 = ex2(s0.x - ref), f1 = ex2(s1.x - ref);
        const float lsum = s0.y * f0 + s1.y * f1;
        const int gr = seg.rt * kR + row;
        const bool live = row < seg.rows;
        const float inv = seg.whole ? (lsum == 0.0f ? 0.0f : 1.0f / lsum) : 1.0f;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (seg.t0 > 0 ? 0 : 1);
        const bool poison = *reinterpret_cast<volatile int*>(&sh.poison) != 0;
        const uint32_t o0 = tm + lanes + 256 + w * (D / 2), o1 = o0 + 128;
#pragma unroll 1
        for (int i = 0; i < D / 64; ++i) {
          float x[32];
          __syncwarp();
          tc_ld32(o0 + i * 32, x);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = s0.x == -INFINITY ? 0.0f : x[k] * f0;
          if (n > 1) {
            float y[32];
            tc_ld32(o1 + i * 32, y);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] += s1.x == -INFINITY ? 0.0f : y[k] * f1;
          }
          const int d0 = w * (D / 2) + i * 32;
          if (live) {
            if (seg.whole) {
              T* out = static_cast<T*>(a.out) +
                       ((seg.q.first + gr / group) * a.q_heads + seg.h * group + gr % group) * (int64_t)D + d0;
#pragma unroll
              for (int k = 0; k < 32; k += 8)
                *reinterpret_cast<uint4*>(out + k) =
                    make_uint4(pack2(x[k] * inv, x[k + 1] * inv, T()), pack2(x[k + 2] * inv, x[k + 3] * inv, T()),
                               pack2(x[k + 4] * inv, x[k + 5] * inv, T()), pack2(x[k + 6] * inv, x[k + 7] * inv, T()));
            } else {
              float* out = part.sums + (slot * kR + row) * D + d0;
#pragma unroll
              for (int k = 0; k < 32; k += 8) store32(out + k, reinterpret_cast<const uint32_t*>(x + k));
            }
          }
        }
        // values that are not finite were left out of the tiles that hold nodes:
        // the rows that see their keys get them now
        if (poison && live && !gone) {
          T* out = nullptr;
          if (seg.whole)
            out = static_cast<T*>(a.out) + ((seg.q.first + gr / group) * a.q_heads + seg.h * group + gr % group) * (int64_t)D;
          left_out<T, FP8, D>(a.c, seg, gr / group, w * (D / 2), out, part.sums + (slot * kR + row) * D);
        }
        if (live && !seg.whole && w == 0) part.stats[slot * kR + row] = make_float2(mm, gone ? kLostRow : lsum);
      }
      tc_fence_before();
      named_bar_sync(1, kSoftmaxThreads);   // the sums are read before queries lie over them
      if (sid == 0) {
        leave_open(part.open, seg, scan.total, G, group);
        next_segment<kR>(&seg, plan);
      }
      named_bar_sync(1, kSoftmaxThreads);
      tile0 += n;
      ++g;
    }
  }
  if (bad) atomicOr(c.err, bad);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh.dead) {   // copies and products that no role has waited for end before their memory goes
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    if (tid == 0) atomicOr(c.err, SPECDEC_DEVERR_TIMEOUT);
    __syncthreads();
  }
  if (warp == kProductWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(512));
}

template <bool CROSS, typename T, bool FP8, int D>
int launch_tile(const AttendArgs& a, int num_sms, cudaStream_t st) {
  auto kern = attend_tile_kernel<T, FP8, D, CROSS>;
  constexpr int bytes = TileLayout<T, FP8, D>::BYTES;
  static std::atomic<uint64_t> done{0};
  if (!allow_shared(kern, bytes, done)) return SPECDEC_ERR_CUDA;
  // rows of a box: within one page, whole groups of 8 rows of the swizzle
  const int page = a.c.geo.page_size;
  int box = 128;
  while (box > 4 && page % box) box >>= 1;
  if (box < 8) box = 0;
  // scales of 4 keys are read at once
  const bool grouped = box >= 32 && (!FP8 || (reinterpret_cast<uintptr_t>(a.c.ks) % 16 == 0 && reinterpret_cast<uintptr_t>(a.c.vs) % 16 == 0));
  if (!grouped && box > 16) box = 16;
  CUtensorMap kmap = {}, vmap = {};
  const int64_t rows = a.c.geo.num_pages * a.c.geo.kv_heads * page;
  if (box && (!encode_rows(&kmap, a.c.k, rows, D, box, FP8) || !encode_rows(&vmap, a.c.v, rows, D, box, FP8))) box = 0;
  kern<<<num_sms, kTileThreads, bytes, st>>>(a, box, grouped && box > 0, kmap, vmap);
  if (cudaGetLastError() != cudaSuccess) return SPECDEC_ERR_CUDA;
  return a.whole ? SPECDEC_OK : launch_join<T, kR, D>(a, num_sms, st);
}

template <bool CROSS, typename T, bool FP8>
int launch_tile_dim(const AttendArgs& a, int num_sms, cudaStream_t st) {
  return a.c.head_dim == 128 ? launch_tile<CROSS, T, FP8, 128>(a, num_sms, st) : launch_tile<CROSS, T, FP8, 64>(a, num_sms, st);
}

template <bool CROSS>
int launch_tile_types(const AttendArgs& a, int cache_dtype, int dtype, int num_sms, cudaStream_t st) {
  const bool fp8 = cache_dtype == SPECDEC_E4M3;
  if (dtype == SPECDEC_BF16)
    return fp8 ? launch_tile_dim<CROSS, __nv_bfloat16, true>(a, num_sms, st)
               : launch_tile_dim<CROSS, __nv_bfloat16, false>(a, num_sms, st);
  return fp8 ? launch_tile_dim<CROSS, __half, true>(a, num_sms, st) : launch_tile_dim<CROSS, __half, false>(a, num_sms, st);
}

}  // namespace
}  // namespace specdec
