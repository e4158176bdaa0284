// Log probabilities of given tokens, with the entropy and the top alternatives of
// their rows, and the gradient of the logits.  Contract in include/specdec.h
// (specdec_logprobs, specdec_logprobs_grad).
//
// With c = log2(e) / T, a reference rho near the row's largest logit and y_v = (x_v - rho) c,
//   S = sum 2^y_v,  W = sum 2^y_v y_v,
//   ln p(v) = ln 2 (y_v - log2 S),  H = ln 2 (log2 S - W / S).
// The difference is taken first: it is exact for neighbouring logits, however large.
//
// One pass over a row, bound by memory where rows are many: 2048 rows of 128256 bf16 90 us,
// 5.8 TB/s (with 20 alternatives 104); 640 of 151936 36 us, 5.4 TB/s (45; all rows in one
// wave of blocks).  Two batches of loads take turns, so that one is always under way; 6
// blocks of an SM instead of 5 took 98 and 40 us, 256 threads in 3 blocks 93 and 43.  Blocks
// that stay and take tokens in turns, finding those with an id by a count, took 93 and 128
// with alternatives; a call of 6400 tokens with 640 ids is no faster that way either (its
// blocks without an id cost 8 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/specdec.h"
#include "device_common.cuh"
#include "logprob.cuh"

namespace specdec {
namespace {

constexpr int kNT = 128, kNW = kNT / 32;   // threads of a row's block
constexpr int kBlocks = 5;                 // of them on an SM
constexpr int kU = 4;                      // 16-byte loads of a thread under way together
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kFloor = -1000.0f;         // y of entries without weight, where they meet a product
constexpr float kLeast = -3.402823466e38f;   // the lowest finite number
constexpr float kLazy = 8.0f;              // log2 of how far the reference may lag behind the largest entry
constexpr int kGroups = 64, kGroup = kNT / kGroups;   // groups of threads, whose largest entries set the bound
constexpr int kRoom = 1024;                // 16-byte pieces that a block puts aside at most
constexpr int kCand = 2 * kNT;             // candidates at most
constexpr int kCap = 96;                   // of a warp's list, where those were too many

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
struct Row;   // what differs between the types of logits (raised, lifted: to at least low, or NaN)

template <>
struct Row<float> {
  static constexpr int E = 4;
  static constexpr uint32_t kNone = 0xFF800000u;   // -inf
  using Low = float;
  static __device__ __forceinline__ Low below(float x) { return x; }
  static __device__ __forceinline__ uint4 raised(const uint4& w, Low low) {
    uint4 v;
    const float* f = reinterpret_cast<const float*>(&w);
    float* g = reinterpret_cast<float*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = max_nan(f[i], low);
    return v;
  }
  static __device__ __forceinline__ float2 lifted(float2 f, Low) { return f; }
  static __device__ __forceinline__ float2 two(const uint4& w, int i) {
    const uint32_t* u = &w.x;
    return make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
  }
  static __device__ __forceinline__ float most(const uint4& w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
};
template <>
struct Row<__nv_bfloat16> {
  static constexpr int E = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;
  using Low = __nv_bfloat162;
  static __device__ __forceinline__ Low below(float x) {
    const __nv_bfloat16 b = __float2bfloat16_rd(x);
    return __nv_bfloat162(b, b);
  }
  static __device__ __forceinline__ uint4 raised(const uint4& w, Low low) {
    uint4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<__nv_bfloat162*>(&v)[i] = __hmax2_nan(reinterpret_cast<const __nv_bfloat162*>(&w)[i], low);
    return v;
  }
  static __device__ __forceinline__ float2 lifted(float2 f, Low) { return f; }
  static __device__ __forceinline__ float2 two(const uint4& w, int i) {
    const uint32_t u = (&w.x)[i];
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
  static __device__ __forceinline__ float most(const uint4& w) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
    return fmaxf(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
};
template <>
struct Row<__half> {
  static constexpr int E = 8;
  static constexpr uint32_t kNone = 0xFC00FC00u;
  using Low = float;   // f16 does not reach far enough below its values
  static __device__ __forceinline__ Low below(float x) { return x; }
  static __device__ __forceinline__ uint4 raised(const uint4& w, Low) { return w; }
  static __device__ __forceinline__ float2 lifted(float2 f, Low low) { return make_float2(max_nan(f.x, low), max_nan(f.y, low)); }
  static __device__ __forceinline__ float2 two(const uint4& w, int i) {
    return __half22float2(reinterpret_cast<const __half2*>(&w)[i]);
  }
  static __device__ __forceinline__ float most(const uint4& w) {
    const __half2* h = reinterpret_cast<const __half2*>(&w);
    const float2 f = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
    return fmaxf(f.x, f.y);
  }
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void as_type(float x, float& y) { y = x; }
__device__ __forceinline__ void as_type(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void as_type(float x, __half& y) { y = __float2half_rn(x); }

// Two 32-bit operations in one instruction, each rounded as alone.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Rows are read once: they shall not displace what others keep in the caches.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// ---- sums of a part of a row ---------------------------------------------------

struct Sums {
  float rho, s, w;
};

// Brings the sums to another reference (at least their own, or any for empty sums).
__device__ __forceinline__ void move_to(Sums& a, float rho, float c) {
  if (a.rho == rho) return;
  if (a.rho == -INFINITY) {
    a.s = a.w = 0.0f;
  } else {
    const float d = (a.rho - rho) * c, f = ex2(d);
    a.w = f > 0.0f ? f * fmaf(d < kFloor ? kFloor : d, a.s, a.w) : 0.0f;   // (w: see the end of the kernel)
    a.s *= f;
  }
  a.rho = rho;
}

// All lanes' sums, in every lane.
__device__ __forceinline__ Sums warp_join(Sums a, float c) {
  float rho = a.rho;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float b = __shfl_xor_sync(0xFFFFFFFFu, rho, o);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(rho) : "f"(b));
  }
  move_to(a, rho, c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, o);
    a.w += __shfl_xor_sync(0xFFFFFFFFu, a.w, o);
  }
  return a;
}

// ---- the largest entries of a row -----------------------------------------------
// Entries are ordered by key: the value, then the lower index.  A block takes a bound, a
// value that n of its entries reach, from the largest entries of its 64 groups of threads
// (the n-th largest of 64: a little below the n-th of all that they have seen), and takes
// a new one whenever three times as many batches have gone by.  What reaches the bound
// is put aside as the 16 bytes that hold it, about 10 n of them for a row in no order, and
// looked at by all threads together when the row is through (entries looked at and keys
// made by the thread that meets them, and one bound for the row: 238 us where this form
// took 63, 640 rows of 151936 and n = 20).  Rows of many equal
// entries, of a rising order or with fewer than n entries above -inf leave too many
// candidates or too few: the block then goes over its part again with a list for each warp
// (offer).

__device__ __forceinline__ uint32_t order_of(float x) {   // -0 counts as 0
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) { return (uint64_t)order_of(x) << 32 | (uint32_t)~index; }

__device__ __forceinline__ uint64_t warp_most(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

// The n largest of cnt <= kCap keys in buf, sorted, to buf; how many there are.
__device__ __forceinline__ int keep_most(uint64_t* buf, int cnt, int n) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  uint64_t k[kCap / 32];
#pragma unroll
  for (int i = 0; i < kCap / 32; ++i) k[i] = i * 32 + lane < cnt ? buf[i * 32 + lane] : 0;
  __syncwarp();
  const int m = min(cnt, n);
  for (int r = 0; r < m; ++r) {
    uint64_t mine = k[0];
#pragma unroll
    for (int i = 1; i < kCap / 32; ++i) mine = mine > k[i] ? mine : k[i];
    const uint64_t best = warp_most(mine);
#pragma unroll
    for (int i = 0; i < kCap / 32; ++i)
      if (k[i] == best) k[i] = 0;
    if (lane == 0) buf[r] = best;
  }
  __syncwarp();
  return m;
}

// The least value that may still be among the n largest: a warp looks at entries of
// rising index, so of the value of its list's n-th none can follow, and `known` is the
// order of a value that n entries of the block's part are known to reach (when depends
// on the run, what is found does not).
__device__ __forceinline__ float bound_of(uint32_t own, const volatile uint32_t* known) {
  const uint32_t k = *known;
  return value_of(own > k ? own : k);
}

struct Listed {
  int cnt;        // entries of the warp's list
  uint32_t own;   // order of the least value that its own entries leave room for
};

// Offers the first m of the neighbouring entries in w, the first one's index given.
template <typename T>
__device__ __noinline__ Listed offer(uint64_t* buf, Listed s, int n, uint4 w, int m, uint32_t index, uint32_t* known) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < Row<T>::E; ++i) {
    const float2 f = Row<T>::two(w, i >> 1);
    const float x = i & 1 ? f.y : f.x;
    const bool in = i < m && x >= bound_of(s.own, known);
    const unsigned who = __ballot_sync(0xFFFFFFFFu, in);
    if (!who) continue;
    if (s.cnt + 32 > kCap) {
      // entries of this step may still equal the last one's value with a lower index
      s.cnt = keep_most(buf, s.cnt, n);
      if (lane == 0) atomicMax(known, (uint32_t)(buf[n - 1] >> 32));
      __syncwarp();
    }
    if (in) buf[s.cnt + __popc(who & ((1u << lane) - 1u))] = key_of(x, index + i);
    s.cnt += __popc(who);
  }
  if (s.cnt > n + 32) {
    s.cnt = keep_most(buf, s.cnt, n);
    const uint32_t last = (uint32_t)(buf[n - 1] >> 32);
    s.own = last + 1u;
    if (lane == 0) atomicMax(known, last);
  }
  __syncwarp();
  return s;
}

struct LogprobShared {
  alignas(16) uint4 aside[kRoom];       // pieces with an entry that reached the bound,
  uint32_t index[kRoom];                // and their first entries
  alignas(16) float groups[kGroups];    // read 16 bytes at a time
  Sums part[kNW];
  Sums ranks[8];                        // of the cluster's blocks (rank 0)
  uint32_t known;
  int pieces, found;                    // put aside, and candidates: also those beyond the room
  float bound;
  uint64_t best[kMaxTop];
  uint64_t bests[8 * kMaxTop];          // of the cluster's blocks (rank 0)
  uint64_t cand[kCand];
  uint64_t list[kNW][kCap];
};

// The n largest of cnt keys, in order, to out, by all threads: a thread counts the keys
// above its own.  (Not for cnt > kNT x 2; keys are distinct.)
__device__ __forceinline__ void place_most(const uint64_t* keys, int cnt, int n, uint64_t* out) {
  const int i0 = threadIdx.x, i1 = threadIdx.x + kNT;
  const uint64_t k0 = i0 < cnt ? keys[i0] : 0, k1 = i1 < cnt ? keys[i1] : 0;
  int r0 = 0, r1 = 0;
  if (cnt <= kNT) {
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) r0 += keys[i] > k0;
  } else {
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
      const uint64_t k = keys[i];
      r0 += k > k0;
      r1 += k > k1;
    }
  }
  if (k0 && r0 < n) out[r0] = k0;
  if (k1 && r1 < n) out[r1] = k1;
}

__device__ __forceinline__ void put_remote(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void put_remote(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A token's row, by a cluster of 1, 2, 4 or 8 blocks that take a part of it each; rank
// 0 joins the parts and writes.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kNT, kBlocks) logprob_kernel(const LogprobArgs a) {
  using R = Row<T>;
  constexpr int E = R::E;
  __shared__ LogprobShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int64_t t = blockIdx.x / (unsigned)ranks;
  const int n = a.top;
  const int32_t id = a.ids ? a.ids[t] : 0;
  const int64_t row = a.rows ? (int64_t)a.rows[t] : t;
  if (id < 0 || id >= a.V || row < 0 || row >= a.R) {   // no row is read; the whole cluster leaves
    if (rank == 0) {
      if (tid == 0) {
        if (id >= a.V) atomicOr(a.err, SPECDEC_DEVERR_BAD_DRAFT_ID);
        else if (id >= 0) atomicOr(a.err, SPECDEC_DEVERR_BAD_CU);
        if (a.logprob) a.logprob[t] = 0.0f;
        if (a.entropy) a.entropy[t] = 0.0f;
        if (a.stats) a.stats[t] = make_float2(0.0f, 0.0f);
      }
      if (TOP && tid < n) {
        a.top_ids[t * n + tid] = -1;
        a.top_logprobs[t * n + tid] = 0.0f;
      }
    }
    return;
  }
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this block runs
  const T* x = static_cast<const T*>(a.x) + row * a.row_stride;
  const int lead = min(a.V, (int)((16u - ((uint32_t)reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / (int)sizeof(T));
  const int vecs = (a.V - lead) / E, done = lead + vecs * E;
  const int v0 = (int)((int64_t)vecs * rank / ranks), v1 = (int)((int64_t)vecs * (rank + 1) / ranks);
  const uint4* xv = reinterpret_cast<const uint4*>(x + lead);
  // entries before the first 16-byte boundary and behind the last: the first and last rank's
  const int before = rank == 0 ? lead : 0, behind = rank == ranks - 1 ? a.V - done : 0;
  const float given = a.logprob && rank == 0 && tid == 0 ? as_float(x[id]) : 0.0f;
  if (TOP && tid == 0) {   // (the first bound's barrier follows)
    sh.pieces = sh.found = 0;
    sh.bound = kLeast;
  }
  if (TOP && tid < kMaxTop) sh.best[tid] = 0;
  Sums mine = {-INFINITY, 0.0f, 0.0f};
  uint64_t s2[2] = {0, 0}, w2[2] = {0, 0};
  const uint64_t c2 = pair(a.c, a.c);
  const float lag = kLazy / a.c;
  float ref = 0.0f;
  typename R::Low low = R::below(kFloor / a.c);   // entries of -inf count as this: 0 x -inf would be NaN
  [[maybe_unused]] float bound = kLeast;   // always above -inf, which is never put aside
  auto gather = [&] {
    float p, q;
    unpair(add2(s2[0], s2[1]), p, q);
    mine.s = p + q;
    unpair(add2(w2[0], w2[1]), p, q);
    mine.w = p + q;
  };
  auto most_of = [&](const uint4* w, auto count) {
    float most = R::most(w[0]);
#pragma unroll
    for (int u = 1; u < decltype(count)::value; ++u) most = fmaxf(most, R::most(w[u]));
    return most;
  };
  // U x 16 bytes of a thread; the first one's first index, and how far the others' lie apart
  auto take = [&](const uint4* w, auto count, float most, uint32_t index, uint32_t apart) {
    constexpr int U = decltype(count)::value;
    if (!(most <= mine.rho + lag)) {          // first entries, larger ones, NaN
      gather();
      move_to(mine, most, a.c);
      s2[0] = pair(mine.s, 0.0f);
      w2[0] = pair(mine.w, 0.0f);
      s2[1] = w2[1] = 0;
      ref = -mine.rho;
      // far enough below that 2^y is 0, however rho is rounded
      low = R::below(mine.rho - fmaxf(-kFloor / a.c, fabsf(mine.rho) * 0.03125f));
    }
    const uint64_t r2 = pair(ref, ref);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint4 v = R::raised(w[u], low);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 f = R::lifted(R::two(v, i), low);
        float y0, y1;
        const uint64_t y2 = mul2(add2(pair(f.x, f.y), r2), c2);
        unpair(y2, y0, y1);
        const uint64_t e2 = pair(ex2(y0), ex2(y1));
        s2[i & 1] = add2(s2[i & 1], e2);
        w2[i & 1] = fma2(e2, y2, w2[i & 1]);
      }
    }
    if (TOP && most >= bound) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (R::most(w[u]) >= bound) {
          const int at = atomicAdd(&sh.pieces, 1);
          if (at < kRoom) {
            sh.aside[at] = w[u];
            sh.index[at] = index + u * apart;
          }
        }
    }
  };
  // A bound from what the threads have seen: a group's threads find the place of their
  // largest entry among the others'.
  auto new_bound = [&](float seen) {
#pragma unroll
    for (int o = 1; o < kGroup; o <<= 1) seen = fmaxf(seen, __shfl_xor_sync(0xFFFFFFFFu, seen, o));
    if (tid % kGroup == 0) sh.groups[tid / kGroup] = seen;
    __syncthreads();
    int above = 0, reach = 0;
#pragma unroll
    for (int i = 0; i < kGroups / kGroup; i += 4) {
      const float4 k = *reinterpret_cast<const float4*>(&sh.groups[tid % kGroup * (kGroups / kGroup) + i]);
      above += (k.x > seen) + (k.y > seen) + (k.z > seen) + (k.w > seen);
      reach += (k.x >= seen) + (k.y >= seen) + (k.z >= seen) + (k.w >= seen);
    }
    int both = above | reach << 16;
#pragma unroll
    for (int o = 1; o < kGroup; o <<= 1) both += __shfl_xor_sync(0xFFFFFFFFu, both, o);
    if ((both & 0xFFFF) < n && both >> 16 >= n) sh.bound = fmaxf(seen, kLeast);   // the n-th largest
    __syncthreads();
    bound = sh.bound;
  };
  using Many = std::integral_constant<int, kU>;
  using One = std::integral_constant<int, 1>;
  const uint4 none = make_uint4(R::kNone, R::kNone, R::kNone, R::kNone);
  // A thread's loads lie a kU-th of the part apart: the first ones, which set the bound,
  // then come from all over it.
  const int steps = (v1 - v0) / (kU * kNT);
  [[maybe_unused]] float seen = -INFINITY;
  int next = 0;                        // the batch behind which the bound is taken anew
  auto load = [&](uint4* w, int s) {
#pragma unroll
    for (int u = 0; u < kU; ++u) w[u] = load_once(xv + v0 + (u * steps + s) * kNT + tid);
  };
  auto batch = [&](const uint4* w, int s) {
    const float most = most_of(w, Many());
    if constexpr (TOP) {
      seen = fmaxf(seen, most);
      if (s == next) {
        new_bound(seen);
        next = 3 * next + 2;
      }
    }
    take(w, Many(), most, (uint32_t)(lead + (v0 + s * kNT + tid) * E), (uint32_t)(steps * kNT * E));
  };
  uint4 wa[kU], wb[kU];                // one batch is under way while the other is taken in
  if (steps > 0) load(wa, 0);
  for (int s = 0; s < steps; s += 2) {
    if (s + 1 < steps) load(wb, s + 1);
    batch(wa, s);
    if (s + 1 < steps) {
      if (s + 2 < steps) load(wa, s + 2);
      batch(wb, s + 1);
    }
  }
  for (int v = v0 + steps * kU * kNT; v < v1; v += kNT) {
    uint4 w = none;
    if (v + tid < v1) w = load_once(xv + v + tid);
    const float most = R::most(w);
    if (TOP && v == v0) new_bound(most);
    take(&w, One(), most, (uint32_t)(lead + (v + tid) * E), 0u);
  }
  if (TOP && v0 == v1) __syncthreads();       // pieces is set
  if (before + behind > 0 && warp == 0) {     // fewer than 16 entries, a piece each
    const int at = lane < before ? lane : done + lane - before;
    uint4 w = none;
    if (lane < before + behind) *reinterpret_cast<T*>(&w) = x[at];
    take(&w, One(), R::most(w), (uint32_t)at, 0u);
  }
  gather();
  mine = warp_join(mine, a.c);
  if (lane == 0) sh.part[warp] = mine;
  __syncthreads();
  if constexpr (TOP) {
    const int pieces = sh.pieces, entries = (v1 - v0) * E + before + behind;
    for (int i = tid; pieces <= kRoom && i < pieces; i += kNT) {
      const uint4 w = sh.aside[i];
      const uint32_t index = sh.index[i];
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float2 f = R::two(w, k >> 1);
        const float e = k & 1 ? f.y : f.x;
        if (e >= bound) {
          const int at = atomicAdd(&sh.found, 1);
          if (at < kCand) sh.cand[at] = key_of(e, index + k);
        }
      }
    }
    __syncthreads();
    const int found = sh.found;
    if (pieces <= kRoom && found <= kCand && found >= min(n, entries)) {
      place_most(sh.cand, found, n, sh.best);
    } else {
      // lists for each warp, of rising indices
      if (tid == 0) sh.known = order_of(-INFINITY);
      __syncthreads();
      Listed lst = {0, 0u};
      if (before > 0 && warp == 0) {
        uint4 w = none;
        if (lane < before) *reinterpret_cast<T*>(&w) = x[lane];
        lst = offer<T>(sh.list[warp], lst, n, w, lane < before ? 1 : 0, (uint32_t)lane, &sh.known);
      }
      for (int v = v0; v < v1; v += kNT) {
        const bool in = v + tid < v1;
        uint4 w = none;
        if (in) w = __ldg(xv + v + tid);
        if (__any_sync(0xFFFFFFFFu, in && R::most(w) >= bound_of(lst.own, &sh.known)))
          lst = offer<T>(sh.list[warp], lst, n, w, in ? E : 0, (uint32_t)(lead + (v + tid) * E), &sh.known);
      }
      if (behind > 0 && warp == 0) {
        uint4 w = none;
        if (lane < behind) *reinterpret_cast<T*>(&w) = x[done + lane];
        lst = offer<T>(sh.list[warp], lst, n, w, lane < behind ? 1 : 0, (uint32_t)(done + lane), &sh.known);
      }
      const int kept = keep_most(sh.list[warp], lst.cnt, n);
      if (lane < n) sh.cand[warp * n + lane] = lane < kept ? sh.list[warp][lane] : 0;
      __syncthreads();
      place_most(sh.cand, kNW * n, n, sh.best);
    }
  }
  if (warp == 0) {
    const Sums empty = {-INFINITY, 0.0f, 0.0f};
    mine = warp_join(lane < kNW ? sh.part[lane] : empty, a.c);
  }
  if (TOP) __syncthreads();
  if (ranks > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every block runs
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t at = mapa(smem_addr(&sh.ranks[rank]), 0);
        put_remote(at, mine.rho);
        put_remote(at + 4, mine.s);
        put_remote(at + 8, mine.w);
      }
      if (TOP && lane < n) put_remote(mapa(smem_addr(&sh.bests[rank * n + lane]), 0), sh.best[lane]);
    }
    cluster_sync_all();
    if (rank) return;
    if (warp == 0) {
      const Sums empty = {-INFINITY, 0.0f, 0.0f};
      mine = warp_join(lane < ranks ? sh.ranks[lane] : empty, a.c);
    }
    if constexpr (TOP) {
      place_most(sh.bests, ranks * n, n, sh.best);
      __syncthreads();
    }
  }
  if (warp) return;
  const bool fine = mine.s > 0.0f && mine.s < INFINITY;   // not: no distribution
  // y of entries that are out of reach may pass 32 bits where the reference itself is near
  // their end (0 x inf is NaN); the reference's neighbours are then 2^90 / T and more
  // away, so that it and its equals have all the weight
  if (!(mine.w == mine.w)) mine.w = 0.0f;
  const float none_f = __uint_as_float(0x7FC00000u);
  const float lg = log2f(mine.s);
  if (lane == 0) {
    if (a.logprob) a.logprob[t] = fine ? kLn2 * ((given - mine.rho) * a.c - lg) : none_f;
    if (a.entropy) a.entropy[t] = fine ? kLn2 * (lg - mine.w / mine.s) : none_f;
    if (a.stats) a.stats[t] = fine ? make_float2(mine.rho, lg) : make_float2(none_f, none_f);
  }
  if (TOP && lane < n) {
    const uint64_t k = sh.best[lane];
    const float y = (value_of((uint32_t)(k >> 32)) - mine.rho) * a.c - lg;
    a.top_ids[t * n + lane] = fine && k ? (int32_t)~(uint32_t)k : -1;
    a.top_logprobs[t * n + lane] = !fine ? none_f : k ? kLn2 * y : -INFINITY;
  }
}

// ---- the gradient of the logits ---------------------------------------------------
// With z = log2 p(v) and the gradients g of ln p(id), h of H and g_j of the
// alternatives' ln p:
//   d x_v = (1 / T) (g [v = id] + sum_j g_j [v = id_j] - p (g + sum_j g_j + h (ln p + H)))
// One pass, bound by memory: 921 of 1973 rows of 128257 bf16 (the others are zeros) 117 us,
// 6.3 TB/s; four loads of a thread at a time instead of two 119, eight 132, past the caches
// 123, half or twice the pieces of a block 133 and 131.  The few entries with a term of
// their own are written again, whole, behind the block's.
constexpr int kGT = 256, kGU = 2;
constexpr int kGVecs = 4096;   // 16-byte pieces of a row that a block takes, about

template <typename T>
__global__ void __launch_bounds__(kGT) logprob_grad_kernel(const LogprobGradArgs a, const int parts) {
  using R = Row<T>;
  constexpr int E = R::E;
  const int tid = threadIdx.x, n = a.top;
  const int64_t t = blockIdx.x / (unsigned)parts;
  const int part = (int)(blockIdx.x - (unsigned)t * (unsigned)parts);
  const T* x = static_cast<const T*>(a.x) + t * a.row_stride;
  T* out = static_cast<T*>(a.out) + t * a.out_stride;
  const int32_t id = a.ids ? a.ids[t] : -1;
  const bool live = a.ids ? id >= 0 && id < a.V : true;
  const int lead = min(a.V, (int)((16u - ((uint32_t)reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / (int)sizeof(T));
  const int vecs = (a.V - lead) / E;
  const int v0 = (int)((int64_t)vecs * part / parts), v1 = (int)((int64_t)vecs * (part + 1) / parts);
  // this block's entries
  const int e0 = part ? lead + v0 * E : 0, e1 = part == parts - 1 ? a.V : lead + v1 * E;
  uint4* ov = reinterpret_cast<uint4*>(out + lead);
  if (!live) {
    for (int v = v0 + tid; v < v1; v += kGT) ov[v] = make_uint4(0, 0, 0, 0);
    T zero;
    as_type(0.0f, zero);
    if (part == 0 && tid < lead) out[tid] = zero;
    for (int i = lead + v1 * E + tid; i < e1; i += kGT) out[i] = zero;
    return;
  }
  const float2 st = a.stats[t];
  const float g = a.g_logprob && a.ids ? a.g_logprob[t] : 0.0f, h = a.g_entropy ? a.g_entropy[t] : 0.0f;
  float all = g;
  if (a.g_top)
    for (int j = 0; j < n; ++j) {
      const int32_t at = a.top_ids[t * n + j];
      if (at >= 0 && at < a.V) all += a.g_top[t * n + j];
    }
  const float k0 = -(all + (h != 0.0f ? h * a.entropy[t] : 0.0f)) * a.inv_t, k1 = -h * kLn2 * a.inv_t;
  auto slope = [&](float z) { return ex2(z) * fmaf(k1, fmaxf(z, kFloor), k0); };
  auto one = [&](T v) -> T {
    T y;
    as_type(slope(fmaf(as_float(v) - st.x, a.c, -st.y)), y);
    return y;
  };
  if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
    const uint4* xv = reinterpret_cast<const uint4*>(x + lead);
    const uint64_t c2 = pair(a.c, a.c), r2 = pair(-st.x, -st.x), l2 = pair(-st.y, -st.y), k1_2 = pair(k1, k1), k0_2 = pair(k0, k0);
    auto turn = [&](uint4 w) -> uint4 {
      uint4 y;
      T* to = reinterpret_cast<T*>(&y);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 f = R::two(w, i);
        float z0, z1, b0, b1;
        unpair(fma2(add2(pair(f.x, f.y), r2), c2, l2), z0, z1);
        unpair(fma2(k1_2, pair(fmaxf(z0, kFloor), fmaxf(z1, kFloor)), k0_2), b0, b1);
        as_type(ex2(z0) * b0, to[2 * i]);
        as_type(ex2(z1) * b1, to[2 * i + 1]);
      }
      return y;
    };
    int v = v0;
    for (; v + kGU * kGT <= v1; v += kGU * kGT) {
      uint4 w[kGU];
#pragma unroll
      for (int u = 0; u < kGU; ++u) w[u] = xv[v + u * kGT + tid];   // (out may be x)
#pragma unroll
      for (int u = 0; u < kGU; ++u) ov[v + u * kGT + tid] = turn(w[u]);
    }
    for (; v + tid < v1; v += kGT) ov[v + tid] = turn(xv[v + tid]);
    if (part == 0 && tid < lead) out[tid] = one(x[tid]);
    const int i = lead + v1 * E + tid;
    if (i < e1) out[i] = one(x[i]);
  } else {
    for (int i = e0 + tid; i < e1; i += kGT) out[i] = one(x[i]);
  }
  if (!(a.g_logprob && a.ids) && !a.g_top) return;
  __syncthreads();
  if (tid <= n) {
    const bool own = tid == n;
    const int32_t at = own ? (a.g_logprob ? id : -1) : a.g_top ? a.top_ids[t * n + tid] : -1;
    if (at >= e0 && at < e1) {
      float add = a.g_logprob && at == id ? g : 0.0f;
      if (a.g_top)
        for (int j = 0; j < n; ++j)
          if (a.top_ids[t * n + j] == at) add += a.g_top[t * n + j];
      const float z = (own ? a.logprob[t] : a.top_logprobs[t * n + tid]) * 1.44269504088896341f;
      as_type(fmaf(add, a.inv_t, slope(z)), out[at]);
    }
  }
}

template <typename T>
int forward_of(const LogprobArgs& a, int num_sms, cudaStream_t st) {
  // Blocks of a row: 2 or 4 where the SMs hold them all at once, of at least two loads a
  // thread, and 8 where they fill two thirds of the SMs at most.  us of 1, 2, 4, 8 blocks a
  // row, none and 20 alternatives: rows of 128256 bf16
  //   48   - - 8.3 7.3, - - 13.7 13.4      152  19.6 13.4 12.4 14.5, 23.6 18.6 19.6 27.2
  //   64   - - 8.3 7.3, - - 14.5 15.5      380  25.7 20.6 30.9 37.1, 30.0 27.7 43.9 60.4
  //   95   15.5 10.1 8.6 11.4, 20.6 17.3 15.5 20.8      1000  55 53 66 87, 62 70 95 142
  const int vecs = a.V / Row<T>::E;
  const int64_t slots = (int64_t)kBlocks * num_sms;
  int ranks = 1;
  while (ranks < 8 && (ranks < 4 ? 2 * a.M * ranks <= slots : 12 * a.M <= slots) && vecs / (2 * ranks) >= 2 * kNT) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.M * ranks));
  cfg.blockDim = dim3(kNT);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.top ? cudaLaunchKernelEx(&cfg, logprob_kernel<T, true>, a) : cudaLaunchKernelEx(&cfg, logprob_kernel<T, false>, a);
  return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

template <typename T>
int gradient_of(const LogprobGradArgs& a, cudaStream_t st) {
  const int64_t vecs = a.V / Row<T>::E;
  int64_t parts = (vecs + kGVecs - 1) / kGVecs;
  if (parts < 1) parts = 1;
  while (parts > 1 && a.M * parts > INT32_MAX) --parts;
  logprob_grad_kernel<T><<<(unsigned)(a.M * parts), kGT, 0, st>>>(a, (int)parts);
  return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace

int launch_logprob(const LogprobArgs& a, int dtype, int num_sms, cudaStream_t st) {
  if (a.M == 0) return SPECDEC_OK;
  if (dtype == SPECDEC_F32) return forward_of<float>(a, num_sms, st);
  return dtype == SPECDEC_BF16 ? forward_of<__nv_bfloat16>(a, num_sms, st) : forward_of<__half>(a, num_sms, st);
}

int launch_logprob_grad(const LogprobGradArgs& a, int dtype, int num_sms, cudaStream_t st) {
  if (a.M == 0) return SPECDEC_OK;
  if (dtype == SPECDEC_F32) return gradient_of<float>(a, st);
  return dtype == SPECDEC_BF16 ? gradient_of<__nv_bfloat16>(a, st) : gradient_of<__half>(a, st);
}

}  // namespace specdec
