// Attention of drafted nodes (chains and token trees) over the paged cache.
// Contract in include/specdec.h (specdec_tree_attention).
//
// attend_warp_kernel: few rows per request (16 a tile).  The pass is
// bound by reading the cache once; each warp streams its own 16 or 32 keys of
// a tile through a ring in shared memory (asynchronous 16-byte copies, three
// blocks deep, no block-wide barrier), keeps the running maximum, sum and
// weighted sum of its keys in registers, and the warps meet once per segment.
// Measured (32 query and 8 kv heads of 128, bf16): one node over 500 keys 12 us, all
// of it latency; 64 nodes over up to 4000 keys 593 MB in 111 us, 5.4 TB/s, the copies
// of a CTA not deep enough at its first and last blocks (70 % of DRAM's cycles).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention.cuh"

namespace specdec {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kRowsTile = 16;   // rows of an item's tile: one mma.sync

template <bool FP8, int D>
struct WarpTile {
  static constexpr int KB = (FP8 || D == 64) ? 32 : 16;        // keys of a warp's block
  static constexpr int TK = KB * kWarps;                       // keys of a unit
  static constexpr int ROW = D * (FP8 ? 1 : 2);                // bytes of a cache row
  static constexpr int CH = ROW / 16;                          // 16-byte chunks of a row
  static constexpr int STAGE = 2 * KB * ROW + (FP8 ? 2 * KB * 4 : 0);
  static constexpr int RING = kWarps * kStages * STAGE;
};

template <bool FP8, int D, int R>
struct WarpLayout {
  using W = WarpTile<FP8, D>;
  static constexpr int MERGE = kWarps * R * (D * 4 + 8);       // reuses the ring
  static constexpr int Q = W::RING > MERGE ? W::RING : MERGE;  // R rows of D 16-bit values
  static constexpr int ROWF = Q + R * D * 2;                   // per-row factor of the scores
  static constexpr int ANC = ROWF + R * 4;                     // ancestors of the tile's nodes
  static constexpr int BYTES = ANC + R * (kMaxTreeNodes / 8);
};

// Chunk c of row r, spread so that 8 rows of one chunk lie in different banks.
template <int CH>
__device__ __forceinline__ int spread(int r, int c) {
  if constexpr (CH == 4) return r * CH + (c ^ ((r >> 1) & 3));
  else return r * CH + (c ^ (r & 7));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, __half) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The largest weight is 2^kHeadroom: f16 weights keep their 11 bits down to
// 2^-24 of the largest (2^-14 otherwise); bf16 has the exponents anyway.  Sums
// and weighted sums carry the factor alike.
template <typename E>
constexpr float kHeadroom = std::is_same<E, __half>::value ? 10.0f : 0.0f;

// Two e4m3 values (the low 16 bits of w) as f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Element d of key `key` of a V block, as stored (an 8-bit one without scale).
template <typename T, bool FP8, int CH>
__device__ __forceinline__ float v_element(const char* v, int key, int d) {
  if constexpr (FP8) {
    const uint8_t x = static_cast<uint8_t>(v[spread<CH>(key, d / 16) * 16 + d % 16]);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(x, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  } else {
    return to_float(reinterpret_cast<const T*>(v + spread<CH>(key, d / 8) * 16)[d % 8]);
  }
}

// Bits of the non-finite elements of a 16-byte chunk of V (one per element).
template <typename T, bool FP8>
__device__ __forceinline__ uint32_t nonfinite(uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t got = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (FP8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) got |= (uint32_t)(((u[i] >> (8 * k)) & 0x7Fu) == 0x7Fu) << (4 * i + k);
    } else {
      constexpr uint32_t E = sizeof(T) == 2 && std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
#pragma unroll
      for (int k = 0; k < 2; ++k) got |= (uint32_t)(((u[i] >> (16 * k)) & E) == E) << (2 * i + k);
    }
  }
  return got;
}

template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_warp_kernel(const AttendArgs a) {
  using W = WarpTile<FP8, D>;
  using E = typename std::conditional<FP8, __half, T>::type;   // type of the products' factors
  constexpr int R = kRowsTile, KB = W::KB, TK = W::TK, CH = W::CH;
  using L = WarpLayout<FP8, D, R>;
  constexpr int QCH = D / 8;
  extern __shared__ __align__(128) char smem[];
  __shared__ ScanShared scan;
  __shared__ int lost[R];           // nodes of the tile whose parents do not lead to node 0
  const CacheArgs& c = a.c;
  const int G = gridDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.q_heads / c.geo.kv_heads;
  const PlanArgs plan(a);
  uint32_t why = 0;
  int64_t u0 = 0;
  find_unit<kThreads>(plan, R, TK,
                      [&](int64_t units) {
                        const int ranges = (int)min((int64_t)G, units);
                        u0 = (int)blockIdx.x < ranges ? range_begin(units, ranges, blockIdx.x) : units;
                        return u0;
                      },
                      scan, why);
  if (blockIdx.x == 0 && why) atomicOr(c.err, why);
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t units = scan.total;
  const int ranges = (int)min((int64_t)G, units);
  if ((int)blockIdx.x >= ranges || scan.b < 0) return;
  const int64_t uend = range_begin(units, ranges, blockIdx.x + 1);
  const Partials<R, D> part(a.workspace, G);
  int b = scan.b;
  int64_t base = scan.before;       // units before request b
  char* ring = smem + warp * (kStages * W::STAGE);
  const uint32_t ring_s = smem_addr(ring);
  const uint32_t q_s = smem_addr(smem + L::Q);
  float* rowf = reinterpret_cast<float*>(smem + L::ROWF);
  uint32_t* anc = reinterpret_cast<uint32_t*>(smem + L::ANC);
  const int quad = lane & 3, qrow = lane >> 2;
  uint32_t bad = 0;

  uint32_t ignored = 0;
  Request q = attend_request(plan, b, R, TK, ignored);
  for (int64_t u = u0; u < uend;) {
    while (u >= base + q.units) {
      base += q.units;
      if (++b >= c.B) return;   // lengths that changed under the call
      q = attend_request(plan, b, R, TK, ignored);
    }
    const int cost = (a.whole ? 1 : q.tiles) + plan.item_cost;
    const int64_t item = (u - base) / cost;
    const int at = (int)((u - base) % cost);
    const int t0 = max(at - plan.item_cost, 0);
    int t1 = (int)min((int64_t)(cost - plan.item_cost), at - plan.item_cost + (uend - u));
    const int h = (int)(item / q.rts), rt = (int)(item % q.rts);
    u += cost - at;
    if (t1 <= t0) continue;
    if (a.whole) t1 = q.tiles;
    const bool whole = t0 == 0 && t1 == q.tiles;
    const int rows = min(R, q.n * group - rt * R);            // rows of this tile
    const int node0 = rt * R / group;                          // its first node
    const int32_t* pages = c.table + b * c.geo.table_stride;
    const int32_t* parent = c.parent ? c.parent + q.first : nullptr;
    const int words = (q.n + 31) >> 5;

    __syncthreads();   // the last segment's readers are done
    // ---- the warp's blocks: tile t, keys [t TK + warp KB, + KB) --------------
    const int64_t all_keys = (int64_t)q.len + q.n;
    auto row_of = [&](int t) -> int {   // cache row of this lane's key of block t, -1: none
      const int64_t s = (int64_t)t * TK + warp * KB + lane;
      if (t >= t1 || lane >= KB || s >= all_keys) return -1;
      const int64_t r = cache_row(c.geo, pages, s);
      if (r < 0) {
        bad |= SPECDEC_DEVERR_BAD_CACHE;
        return -1;
      }
      return (int)(r + (int64_t)h * c.geo.page_size);
    };
    auto issue = [&](int t, int row) {
      const uint32_t st = ring_s + ((t - t0) % kStages) * W::STAGE;
      if (t < t1) {
#pragma unroll
        for (int i = 0; i < KB * CH / 32; ++i) {
          const int x = i * 32 + lane, key = x / CH, ch = x % CH;
          const int r = __shfl_sync(0xFFFFFFFFu, row, key);
          const int64_t off = (int64_t)max(r, 0) * W::ROW + ch * 16;
          const uint32_t dst = st + spread<CH>(key, ch) * 16;
          copy16(dst, static_cast<const char*>(c.k) + off, r >= 0);
          copy16(dst + KB * W::ROW, static_cast<const char*>(c.v) + off, r >= 0);
        }
        if constexpr (FP8) {
          copy4(st + 2 * KB * W::ROW + lane * 4, c.ks + max(row, 0), row >= 0);
          copy4(st + 2 * KB * W::ROW + KB * 4 + lane * 4, c.vs + max(row, 0), row >= 0);
        }
      }
      copy_commit();
    };
    int rows_now[kStages];            // cache rows of the blocks in flight (which keys are live)
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      rows_now[i] = row_of(t0 + i);
      issue(t0 + i, rows_now[i]);
    }
    int ahead = row_of(t0 + kStages - 1);
    // ---- queries: shared memory, as the products want them (the first blocks are
    // on their way meanwhile) ---------------------------------------------------
    for (int r = warp; r < R; r += kWarps) {
      constexpr int PER = D / 32;
      float x[PER];
      const int row = rt * R + r;
      const bool live = r < rows;
      const T* src = static_cast<const T*>(a.q) + (q.first + (live ? row / group : 0)) * a.q_row +
                     (int64_t)(h * group + (live ? row % group : 0)) * a.q_head + lane * PER;
#pragma unroll
      for (int k = 0; k < PER; ++k) x[k] = live ? to_float(src[k]) : 0.0f;
      float f = a.scale_log2;
      if constexpr (FP8) {
        // f16 factors: the row is scaled by a power of two so that its largest
        // value lies in [1, 2); the scores take the factor back
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < PER; ++k) m = fmaxf(m, fabsf(x[k]));
        m = warp_max(m);
        const int e = min(max((int)(__float_as_uint(m) >> 23), 1), 253);
        const float mul = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
        for (int k = 0; k < PER; ++k) x[k] *= mul;
        f *= __uint_as_float((uint32_t)e << 23);
      }
      if (lane == 0) rowf[r] = f;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        int d = lane * PER + k;
        if constexpr (FP8) {
          // a key's 4 neighbouring bytes feed the two halves of a lane's
          // factor: d = 16 i + 4 j + k goes to 16 i + 2 j + k, or + 8 for k > 1
          const int i = d & 15, j = i >> 2, s = i & 3;
          d = (d & ~15) + (s < 2 ? 2 * j + s : 6 + 2 * j + s);
        }
        E y;
        from_float(x[k], y);
        reinterpret_cast<E*>(smem + L::Q + spread<QCH>(r, d / 8) * 16)[d % 8] = y;
      }
    }
    const bool tail = (int64_t)t1 * TK > q.len;                // the segment sees nodes
    if (tail && parent) {
      const int nodes = (rt * R + rows - 1) / group - node0 + 1;
      for (int i = tid; i < nodes; i += kThreads) {
        lost[i] = !ancestor_bits(parent, node0 + i, words, anc + i * words);
        if (lost[i]) bad |= SPECDEC_DEVERR_BAD_TREE;
      }
    }
    __syncthreads();

    float o[D / 8][4];
    float m[2], l[2];
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
#pragma unroll
    for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[nt][k] = 0.0f;
    float rf[2];
    rf[0] = rowf[qrow];
    rf[1] = rowf[qrow + 8];
    for (int t = t0; t < t1; ++t) {
      issue(t + kStages - 1, ahead);
      const int now = rows_now[0];
#pragma unroll
      for (int i = 0; i + 1 < kStages - 1; ++i) rows_now[i] = rows_now[i + 1];
      rows_now[kStages - 2] = ahead;
      ahead = row_of(t + kStages);
      copy_wait<kStages - 1>();
      __syncwarp();
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, now >= 0);
      if (live) {
        const uint32_t k_s = ring_s + ((t - t0) % kStages) * W::STAGE, v_s = k_s + KB * W::ROW;
        char* kv = ring + ((t - t0) % kStages) * W::STAGE;
        float s[KB / 8][4];
#pragma unroll
        for (int nt = 0; nt < KB / 8; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[nt][k] = 0.0f;
        // scores: rows x keys, 16 of the head dimension at a time
#pragma unroll
        for (int kk = 0; kk < D / 16; kk += (FP8 ? 2 : 1)) {
          uint32_t qa[FP8 ? 2 : 1][4];
#pragma unroll
          for (int z = 0; z < (FP8 ? 2 : 1); ++z)
            ldm4(q_s + spread<QCH>(lane & 15, (kk + z) * 2 + (lane >> 4)) * 16, qa[z]);
#pragma unroll
          for (int np = 0; np < KB / 16; ++np) {
            uint32_t w[4];
            const int key = np * 16 + (lane & 7) + ((lane >> 4) << 3);
            const int ch = (FP8 ? kk : kk * 2) + ((lane >> 3) & 1);
            ldm4(k_s + spread<CH>(key, ch) * 16, w);
            if constexpr (FP8) {
#pragma unroll
              for (int i = 0; i < 2; ++i)      // n-tile
#pragma unroll
                for (int z = 0; z < 2; ++z) {  // 16 of the head dimension
                  const uint32_t b0 = e4m3x2_f16x2(w[2 * i + z]), b1 = e4m3x2_f16x2(w[2 * i + z] >> 16);
                  mma16816(s[2 * np + i], qa[z], b0, b1, E());
                }
            } else {
              mma16816(s[2 * np], qa[0], w[0], w[1], E());
              mma16816(s[2 * np + 1], qa[0], w[2], w[3], E());
            }
          }
        }
        // base-2 scores, masks, the block's maximum.  8-bit values carry their
        // scale in the exponent: the weights that meet V are
        // 2^(u + log2 vs - m), whose largest 16 bits hold whatever the scales are
        const int64_t key0 = (int64_t)t * TK + warp * KB;
        const bool masked = live != (KB == 32 ? 0xFFFFFFFFu : (1u << (KB & 31)) - 1u) || key0 + KB > q.len;
        float iv[FP8 ? KB / 8 : 1][2];   // 1 / vs
        float mx[2];
        mx[0] = mx[1] = -INFINITY;
        auto sees = [&](int r, int key) -> bool {
          if (!((live >> key) & 1u)) return false;
          const int64_t j = key0 + key - q.len;
          if (j < 0) return true;
          if (r >= rows) return false;
          const int node = (rt * R + r) / group;
          return parent ? (anc[(node - node0) * words + (int)(j >> 5)] >> (j & 31)) & 1u : j <= node;
        };
#pragma unroll
        for (int nt = 0; nt < KB / 8; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = nt * 8 + quad * 2 + x;
            float kf = 1.0f, lv = 0.0f;
            if constexpr (FP8) {
              kf = reinterpret_cast<const float*>(kv + 2 * KB * W::ROW)[key];
              const float vf = reinterpret_cast<const float*>(kv + 2 * KB * W::ROW + KB * 4)[key];
              // a scale of 0 (a row of zeros) is as good as a very small one
              const float vc = vf == vf ? fmaxf(vf, 8.673617379884035e-19f) : vf;
              lv = __log2f(vc);
              iv[nt][x] = __frcp_rn(vc);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float& e = s[nt][2 * y + x];
              e = FP8 ? fmaf(e * kf, rf[y], lv) : e * rf[y];
              if (masked && !sees(qrow + 8 * y, key)) e = -INFINITY;
              mx[y] = fmaxf(mx[y], e);
            }
          }
        bool moved = false;
        float ref[2], fix[2];   // weights are 2^(e - ref)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float v = mx[y];
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
          const float mn = fmaxf(m[y], v);
          moved |= mn != m[y];
          const float at = mn == -INFINITY ? 0.0f : mn;
          fix[y] = ex2(m[y] - at);
          ref[y] = at - kHeadroom<E>;
          m[y] = mn;
        }
        if (__any_sync(0xFFFFFFFFu, moved)) {
          l[0] *= fix[0];
          l[1] *= fix[1];
#pragma unroll
          for (int nt = 0; nt < D / 8; ++nt) {
            o[nt][0] *= fix[0];
            o[nt][1] *= fix[0];
            o[nt][2] *= fix[1];
            o[nt][3] *= fix[1];
          }
        }
        // weights; rounded to 16 bits for the product with V (at most half a
        // step of a factor in [0, 1] each), summed unrounded
        uint32_t p[KB / 16][4];
#pragma unroll
        for (int nt = 0; nt < KB / 8; ++nt) {
          float w[4];
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float e = ex2(s[nt][2 * y + x] - ref[y]);
              w[2 * y + x] = e;
              if constexpr (FP8) l[y] += s[nt][2 * y + x] == -INFINITY ? 0.0f : e * iv[nt][x];
              else l[y] += e;
            }
          p[nt / 2][(nt & 1) * 2] = pack2(w[0], w[1], E());
          p[nt / 2][(nt & 1) * 2 + 1] = pack2(w[2], w[3], E());
        }
        // A value that is not finite belongs to the rows that see its key and
        // to no other (0 x inf would reach them through the product): it is
        // added to those and taken out of the block.  Only blocks that some
        // row does not see in full need the look.
        if (masked) {
          char* vb = kv + KB * W::ROW;
          uint32_t any = 0;
          for (int x = lane; x < KB * CH; x += 32) any |= nonfinite<T, FP8>(*reinterpret_cast<uint4*>(vb + x * 16));
          if (__any_sync(0xFFFFFFFFu, any)) {
            for (int key = 0; key < KB; ++key)
#pragma unroll
              for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int d = FP8 ? (nt >> 1) * 16 + quad * 4 + (k & 1) * 2 + (nt & 1) : nt * 8 + quad * 2 + (k & 1);
                  const float v = v_element<T, FP8, CH>(vb, key, d);
                  if (!isfinite(v) && sees(qrow + 8 * (k >> 1), key)) o[nt][k] += v;
                }
            __syncwarp();
            for (int x = lane; x < KB * CH; x += 32) {
              const uint32_t got = nonfinite<T, FP8>(*reinterpret_cast<uint4*>(vb + x * 16));
              for (int i = 0; i < (FP8 ? 16 : 8); ++i)
                if ((got >> i) & 1u) {
                  if constexpr (FP8) vb[x * 16 + i] = 0;
                  else reinterpret_cast<uint16_t*>(vb + x * 16)[i] = 0;
                }
            }
            __syncwarp();
          }
        }
        // values: 16 keys at a time
#pragma unroll
        for (int kk = 0; kk < KB / 16; ++kk)
#pragma unroll
          for (int dt = 0; dt < D / 8; dt += (FP8 ? 4 : 2)) {
            uint32_t w[4];
            const int key = kk * 16 + (lane & 15);
            const int ch = (FP8 ? dt / 2 : dt) + (lane >> 4);
            ldm4t(v_s + spread<CH>(key, ch) * 16, w);
            if constexpr (FP8) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // [k0 d0, k0 d1, k1 d0, k1 d1] -> the key pairs of d0, then of d1
                const uint32_t x = __byte_perm(w[2 * i], 0, 0x3120), y = __byte_perm(w[2 * i + 1], 0, 0x3120);
                const uint32_t x0 = e4m3x2_f16x2(x), x1 = e4m3x2_f16x2(x >> 16);
                const uint32_t y0 = e4m3x2_f16x2(y), y1 = e4m3x2_f16x2(y >> 16);
                mma16816(o[dt + 2 * i], p[kk], x0, y0, E());
                mma16816(o[dt + 2 * i + 1], p[kk], x1, y1, E());
              }
            } else {
              mma16816(o[dt], p[kk], w[0], w[1], E());
              mma16816(o[dt + 1], p[kk], w[2], w[3], E());
            }
          }
      }
      __syncwarp();   // the block is read before its stage is filled again
    }
    copy_wait<0>();
    // ---- the warps meet -------------------------------------------------------
    __syncthreads();
    float* merge = reinterpret_cast<float*>(smem);                       // [warps][R][D]
    float2* stats = reinterpret_cast<float2*>(smem + kWarps * R * D * 4);  // [warps][R]
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float v = l[y];
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
      const int r = qrow + 8 * y;
      if (r >= rows) continue;
      if (quad == 0) stats[warp * R + r] = make_float2(m[y], v);
#pragma unroll
      for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int d = FP8 ? (nt >> 1) * 16 + quad * 4 + x * 2 + (nt & 1) : nt * 8 + quad * 2 + x;
          merge[(warp * R + r) * D + d] = o[nt][2 * y + x];
        }
    }
    __syncthreads();
    const int64_t slot = 2 * (int64_t)blockIdx.x + (t0 > 0 ? 0 : 1);
    for (int x = tid; x < rows * D; x += kThreads) {
      const int r = x / D, d = x % D;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, stats[w * R + r].x);
      const float ref = mm == -INFINITY ? 0.0f : mm;
      float sum = 0.0f, acc = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 s = stats[w * R + r];
        const float f = ex2(s.x - ref);
        sum += s.y * f;
        acc += s.x == -INFINITY ? 0.0f : merge[(w * R + r) * D + d] * f;
      }
      const bool gone = tail && parent && lost[(rt * R + r) / group - node0];   // a row of zeros
      if (whole) {
        const int row = rt * R + r;
        T y;
        from_float(gone || sum == 0.0f ? 0.0f : acc / sum, y);
        static_cast<T*>(a.out)[((q.first + row / group) * a.q_heads + h * group + row % group) * (int64_t)D + d] = y;
      } else {
        part.sums[(slot * R + r) * D + d] = acc;
        if (d == 0) part.stats[slot * R + r] = make_float2(mm, gone ? kLostRow : sum);
      }
    }
  }
  if (bad) atomicOr(c.err, bad);
}

template <typename T, bool FP8, int D>
int launch_warp(const AttendArgs& a, int num_sms, cudaStream_t st) {
  using L = WarpLayout<FP8, D, kRowsTile>;
  constexpr int TK = WarpTile<FP8, D>::TK;
  auto kern = attend_warp_kernel<T, FP8, D>;
  static std::atomic<uint64_t> done{0};
  if (!allow_shared(kern, L::BYTES, done)) return SPECDEC_ERR_CUDA;
  const int G = num_sms;
  kern<<<G, kThreads, L::BYTES, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SPECDEC_ERR_CUDA;
  return a.whole ? SPECDEC_OK : launch_join<T, kRowsTile, TK, D>(a, G, st);
}

// Rows (nodes x heads that share a kv head) of an average request: what the
// host knows of the rows of a tile.
int64_t average_rows(int B, int64_t N, int kv_heads, int q_heads) {
  return (N + B - 1) / B * (q_heads / kv_heads);
}
// Up to these (a tile of the warp kernel) the warp kernel, above them the tile kernel.
// One context of 500 / 64 up to 8191 / 4 of 30000 / 200 up to 1500, 8 kv heads of 128,
// device us, warp and tile kernel:
//   4 rows  bf16 11.7 13.7 / 204 211 / 85 89 / 138 177, e4m3 12.7 15.1 / 204 234 / 80 89 / 155 216
//   12      bf16 14.0 13.7 / 213 214 / 89 91 / 165 178, e4m3 14.7 15.4 / 217 241 / 84 91 / 186 219
//   16      bf16 14.8 13.7 / 221 214 / 90 91 / 177 178, e4m3 15.4 15.7 / 224 242 / 85 92 / 195 221
//   20      bf16 15.1 13.7 / 394 217 / 157 92 / 298 179, e4m3 15.7 15.7 / 403 247 / 146 94 / 330 220
// The average decides: in a batch of one large request among many small ones, the
// large one takes a tile of 16 rows at a time.
constexpr int kWarpRows = 16;

template <typename T, bool FP8>
int launch_dim(const AttendArgs& a, int num_sms, cudaStream_t st) {
  return a.c.head_dim == 128 ? launch_warp<T, FP8, 128>(a, num_sms, st) : launch_warp<T, FP8, 64>(a, num_sms, st);
}

}  // namespace

int64_t attend_workspace_bytes(int B, int64_t N, int kv_heads, int q_heads, int head_dim, int64_t capacity, int num_sms) {
  const bool tile = average_rows(B, N, kv_heads, q_heads) > kWarpRows;
  if (whole_items(B, N, kv_heads, q_heads, capacity, tile ? 128 : kRowsTile, num_sms)) return 0;
  if (tile) return attend_tile_workspace(head_dim, num_sms);
  return head_dim == 128 ? Partials<kRowsTile, 128>::bytes(num_sms) : Partials<kRowsTile, 64>::bytes(num_sms);
}

int launch_attend(const AttendArgs& args, int cache_dtype, int dtype, int num_sms, cudaStream_t st) {
  if (args.c.N == 0) return SPECDEC_OK;
  AttendArgs a = args;
  const CacheArgs& c = a.c;
  const bool tile = average_rows(c.B, c.N, c.geo.kv_heads, a.q_heads) > kWarpRows;
  a.whole = whole_items(c.B, c.N, c.geo.kv_heads, a.q_heads, (int64_t)c.geo.max_pages * c.geo.page_size, tile ? 128 : kRowsTile, num_sms);
  const bool fp8 = cache_dtype == SPECDEC_E4M3;
  a.item_cost = fp8 && !tile ? kItemCostWarp8 : kItemCost;
  if (tile) return launch_attend_tile(a, cache_dtype, dtype, num_sms, st);
  if (dtype == SPECDEC_BF16)
    return fp8 ? launch_dim<__nv_bfloat16, true>(a, num_sms, st) : launch_dim<__nv_bfloat16, false>(a, num_sms, st);
  return fp8 ? launch_dim<__half, true>(a, num_sms, st) : launch_dim<__half, false>(a, num_sms, st);
}

}  // namespace specdec
