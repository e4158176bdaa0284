// Verification of drafted chains from target probabilities and given random
// numbers.  Contract in include/specdec.h (specdec_rejection_sample_given).
//
// Only one target row (and, after a rejection, one draft row) of a request is
// read in full: the accept tests need single entries.  The extra token is the
// inverse of the cumulative weights, t = first v with C(v) > s C(V - 1), so the
// sums decide a whole number and are held to about 2^-44, as pairs of floats with
// error-free additions (Knuth, Dekker).  Double precision would be bound by the
// FP64 pipe (two lanes a clock here): even the scans over 64 piece sums and the
// look through the last entries took longer in it than reading the rows.  The errors
// of K additions are themselves summed in 32 bits, which costs (K 2^-24)^2 of the sum
// at the worst, so a lane hands its pair over to a double every 64 additions: 2^-36
// then, whatever V is (additions that all err alike; usual rows come to 2^-44).
//
// A request is a cluster of C CTAs.  Each warp of the cluster sums a contiguous
// piece of the row; the piece sums meet in distributed shared memory (no
// workspace, no atomics, a fixed order); the CTA whose piece holds the crossing
// reads it again, from L2, first by warps and then entry by entry.
//
// Measured: 256 requests of 1 to 8 drafts and 151936 entries, of which 226 reject one
// (two rows each), 293 MB in 59 us = 5.0 TB/s (the accept tests' few dependent loads
// and the final look stand before and after the rows' stream); 8 requests of 32000
// entries 7.6 us, latency.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/specdec.h"
#include "cache.cuh"
#include "device_common.cuh"

namespace specdec {
namespace {

constexpr int kGivenThreads = 256;
constexpr int kGivenWarps = kGivenThreads / 32;
constexpr int kMaxCtas = 8;   // CTAs of a request (the portable cluster size)
constexpr int kMaxPieces = kMaxCtas * kGivenWarps;
constexpr int kStep = 128;   // entries a warp reads at once: 4 per lane
constexpr int kChunk = 4096; // entries that a warp sums in pairs of floats (64 additions a lane)
constexpr int kLook = 16384; // entries that a warp looks through one by one

// Two 32-bit operations in one instruction, each rounded as alone.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {   // a - b: a product with -1 is exact
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(0xBF800000BF800000ull), "l"(a));
  return r;
}

// Two running sums, each hi + lo with |lo| a few roundings of hi (Knuth's two-sum
// gives the error of each addition exactly; lo is not folded into hi on the way).
struct Sums {
  uint64_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(uint64_t w) {
    const uint64_t t = add2(hi, w), b = sub2(t, hi);
    lo = add2(lo, add2(sub2(hi, sub2(t, b)), sub2(w, b)));
    hi = t;
  }
};

// A sum held as hi + lo, |lo| at most half a step of hi.
struct Exact {
  float hi, lo;
};
__device__ __forceinline__ Exact renormed(float s, float e) {   // |s| >= |e|
  const float h = __fadd_rn(s, e);
  return Exact{h, __fsub_rn(e, __fsub_rn(h, s))};
}
__device__ __forceinline__ Exact plus(Exact a, Exact b) {
  const float s = __fadd_rn(a.hi, b.hi), z = __fsub_rn(s, a.hi);
  float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, z)), __fsub_rn(b.hi, z));
  e = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
  return renormed(s, e);
}
__device__ __forceinline__ Exact scaled(Exact a, float s) {
  const float p = __fmul_rn(a.hi, s);
  return renormed(p, __fmaf_rn(a.lo, s, __fmaf_rn(a.hi, s, -p)));
}
__device__ __forceinline__ bool above(Exact a, Exact b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Exact shuffled(Exact a, int from) {
  return Exact{__shfl_sync(0xFFFFFFFFu, a.hi, from), __shfl_sync(0xFFFFFFFFu, a.lo, from)};
}
__device__ __forceinline__ Exact scan_lanes(Exact x, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Exact up = shuffled(x, (lane - o) & 31);
    if (lane >= o) x = plus(up, x);
  }
  return x;
}

// max(0, p - q) with the rounding error of the difference (0 where p <= q).  Where
// p > q >= 0 the error is (p - d) - q, exactly (Dekker).  Entries that are not
// above 0 (NaN among them) weigh nothing.
__device__ __forceinline__ void weigh(float p, float q, float& w, float& e) {
  const float d = __fsub_rn(p, q);
  const float r = __fsub_rn(__fsub_rn(p, d), q);
  const bool on = d > 0.0f;
  w = on ? d : 0.0f;
  e = on ? r : 0.0f;
}

struct Rows {
  const float* p;
  const float* q;   // null: weights are p
  int drop;         // entry whose draft probability is 1 (one-hot drafter), or -1
  int V;
  bool vec;
};

__device__ __forceinline__ void load4(const float* row, int v, int V, bool vec, float* x) {
  if (vec && v + 4 <= V) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(row + v));
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v + k < V ? __ldg(row + v + k) : 0.0f;
  }
}

// One entry's weight and error.
__device__ __forceinline__ void weight(const Rows& R, int v, float p, float q, float& w, float& e) {
  weigh(p, R.q ? q : (v == R.drop ? 1.0f : 0.0f), w, e);
}

// Adds the weights of 4 entries of each of U steps.
template <bool Q, bool WHOLE, int U>
__device__ __forceinline__ void add_steps(const Rows& R, int base, int v1, int lane, Sums& s) {
  float p[U][4], q[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v = base + u * kStep + lane * 4;
    if constexpr (WHOLE) {
      const float4 f = __ldcs(reinterpret_cast<const float4*>(R.p + v));
      p[u][0] = f.x; p[u][1] = f.y; p[u][2] = f.z; p[u][3] = f.w;
      if constexpr (Q) {
        const float4 g = __ldcs(reinterpret_cast<const float4*>(R.q + v));
        q[u][0] = g.x; q[u][1] = g.y; q[u][2] = g.z; q[u][3] = g.w;
      }
    } else if (v < v1) {
      load4(R.p, v, v1, R.vec, p[u]);
      if constexpr (Q) load4(R.q, v, v1, R.vec, q[u]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) p[u][k] = q[u][k] = 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (!Q) {   // a one-hot drafter's entry: max(0, p - 1) in p's place
      const int off = R.drop - (base + u * kStep + lane * 4);
      if ((unsigned)off < 4u) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k == off) p[u][k] = __fsub_rn(p[u][k], 1.0f);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      float w0, w1;
      if constexpr (Q) {
        const uint64_t p2 = pair(p[u][k], p[u][k + 1]), q2 = pair(q[u][k], q[u][k + 1]);
        const uint64_t d2 = sub2(p2, q2);
        float e0, e1;
        unpair(d2, w0, w1);
        unpair(sub2(sub2(p2, d2), q2), e0, e1);
        e0 = w0 > 0.0f ? e0 : 0.0f;
        e1 = w1 > 0.0f ? e1 : 0.0f;
        s.lo = add2(s.lo, pair(e0, e1));
      } else {
        w0 = p[u][k];
        w1 = p[u][k + 1];
      }
      s.add(pair(fmaxf(w0, 0.0f), fmaxf(w1, 0.0f)));   // fmaxf drops NaN
    }
  }
}

// Sum of the weights of [v0, v1) (v0 a multiple of 4) over the warp; LONG: it may pass
// kChunk entries.
template <bool LONG>
__device__ __forceinline__ Exact piece_sum(const Rows& R, int v0, int v1, int lane) {
  constexpr int U = 4;
  double total = 0.0;
  Exact x = {0.0f, 0.0f};
  for (int base = v0; base < v1;) {
    const int end = LONG ? min(v1, base + kChunk) : v1;
    Sums s;
    if (R.vec) {   // whole steps: plain 16-byte loads, all under way before the first is used
      if (R.q) {
        for (; base + U * kStep <= end; base += U * kStep) add_steps<true, true, U>(R, base, v1, lane, s);
      } else {
        for (; base + U * kStep <= end; base += U * kStep) add_steps<false, true, U>(R, base, v1, lane, s);
      }
    }
    if (R.q) {
      for (; base < end; base += U * kStep) add_steps<true, false, U>(R, base, v1, lane, s);
    } else {
      for (; base < end; base += U * kStep) add_steps<false, false, U>(R, base, v1, lane, s);
    }
    float a, b, c, d;
    unpair(s.hi, a, b);
    unpair(s.lo, c, d);
    x = plus(renormed(a, c), renormed(b, d));
    if (!LONG || v1 - v0 <= kChunk) break;   // short pieces stay away from the FP64 pipe
    total += (double)x.hi + (double)x.lo;
  }
  if (LONG && v1 - v0 > kChunk) {
    x.hi = (float)total;
    x.lo = (float)(total - (double)x.hi);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = plus(x, shuffled(x, lane ^ o));
  return x;
}

// First v of [v0, v1) whose cumulative weight (after `before`) is above t;
// the last entry that weighs anything where rounding hides it.
__device__ __forceinline__ int piece_find(const Rows& R, int v0, int v1, Exact before, Exact t, int lane) {
  int last = v0;
  constexpr int U = 4;
  for (int base0 = v0; base0 < v1; base0 += U * kStep) {
    float p[U][4], q[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = base0 + u * kStep + lane * 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) p[u][k] = q[u][k] = 0.0f;
      if (v < v1) {
        load4(R.p, v, v1, R.vec, p[u]);
        if (R.q) load4(R.q, v, v1, R.vec, q[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = base0 + u * kStep + lane * 4;
      if (base0 + u * kStep >= v1) break;
      Exact c[4], sum = {0.0f, 0.0f};
      float w[4], e[4];
      int mine = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        weight(R, v + k, p[u][k], q[u][k], w[k], e[k]);
        sum = plus(sum, Exact{w[k], e[k]});
        c[k] = sum;
        if (w[k] > 0.0f) mine = v + k;
      }
      const Exact scan = scan_lanes(sum, lane);
      Exact at = shuffled(scan, (lane - 1) & 31);
      at = lane ? plus(before, at) : before;
      int hit = -1;
#pragma unroll
      for (int k = 3; k >= 0; --k)
        if (w[k] > 0.0f && above(plus(at, c[k]), t)) hit = v + k;
      const unsigned who = __ballot_sync(0xFFFFFFFFu, hit >= 0);
      if (who) return __shfl_sync(0xFFFFFFFFu, hit, __ffs(who) - 1);
      const unsigned some = __ballot_sync(0xFFFFFFFFu, mine >= 0);
      if (some) last = __shfl_sync(0xFFFFFFFFu, mine, 31 - __clz(some));
      before = plus(before, shuffled(scan, 31));
    }
  }
  return last;
}

__device__ __forceinline__ Exact ld_cluster_sum(uint32_t addr) {
  Exact x;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.hi), "=f"(x.lo) : "r"(addr) : "memory");
  return x;
}

// LONG: a warp's piece of the row passes kChunk entries.  (One kernel for both cost 8
// requests of 32000 entries 0.4 us of 7.9.)
template <bool LONG>
__global__ void __launch_bounds__(kGivenThreads) given_kernel(const GivenArgs a) {
  __shared__ __align__(8) Exact sums[2][kGivenWarps], parts[kGivenWarps];
  const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t d0 = 0;
  int32_t gamma = 0;
  const bool ok = node_range(a.cu, b, a.N_d, d0, gamma);
  // ---- accept tests: 32 positions at a time, the same in every warp ---------
  int n = 0;
  int32_t drop = -1;
  if (ok) {
    bool stopped = false;
    for (int i0 = 0; i0 < gamma && !stopped; i0 += 32) {
      const int i = i0 + lane;
      bool pass = false;
      int32_t x = -1;
      if (i < gamma) {
        x = __ldg(a.ids + d0 + i);
        const float u = __ldg(a.accept_u + d0 + i);
        if (x >= 0 && x < a.V) {
          const float px = __ldg(a.p + (d0 + b + i) * a.p_row + x);
          const float qx = a.q ? __ldg(a.q + (d0 + i) * a.q_row + x) : 1.0f;
          // u < min(1, px / qx) without the division's rounding: 24-bit factors
          // make an exact 48-bit product
          pass = u < 1.0f && (double)u * (double)qx < (double)px;
        } else if (rank == 0 && warp == 0) {
          atomicOr(a.err, SPECDEC_DEVERR_BAD_DRAFT_ID);
        }
      }
      const unsigned fail = __ballot_sync(0xFFFFFFFFu, i < gamma && !pass);
      const int stop = fail ? __ffs(fail) - 1 : 32;
      if (fail) {
        n = i0 + stop;
        stopped = true;
        drop = __shfl_sync(0xFFFFFFFFu, x, stop);
      }
      if (rank == 0 && warp == 0 && i < gamma && lane < stop) a.out_tokens[d0 + b + i] = x;
    }
    if (!stopped) n = gamma;
  } else if (rank == 0 && tid == 0) {
    atomicOr(a.err, SPECDEC_DEVERR_BAD_CU);
  }
  Rows R;
  R.p = a.p + (d0 + b + n) * a.p_row;
  R.q = n < gamma && a.q ? a.q + (d0 + n) * a.q_row : nullptr;
  R.drop = n < gamma && !a.q ? drop : -1;
  R.V = a.V;
  R.vec = a.vec_ok;
  // ---- piece sums; a second round over p alone where the residual is empty --
  const int pieces = C * kGivenWarps;
  const int len = ((a.V + pieces - 1) / pieces + 3) & ~3;
  const int mine = rank * kGivenWarps + warp;
  const int v0 = min(a.V, mine * len), v1 = min(a.V, v0 + len);
  Exact total = {0.0f, 0.0f}, end[kMaxPieces / 32];
  bool heavy_piece[kMaxPieces / 32];
  for (int round = 0; round < 2; ++round) {
    Exact own_sum = {0.0f, 0.0f};
    if (ok) own_sum = piece_sum<LONG>(R, v0, v1, lane);
    if (lane == 0) sums[round][warp] = own_sum;
    cluster_sync_all();
    // the same order in every warp: lane l holds pieces l and l + 32
    total = Exact{0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < kMaxPieces / 32; ++c) {
      end[c] = total;
      heavy_piece[c] = false;
      if (c * 32 >= pieces) continue;
      const int k = c * 32 + lane;
      Exact x = {0.0f, 0.0f};
      if (k < pieces)
        x = ld_cluster_sum(mapa(smem_addr(&sums[round][k % kGivenWarps]), k / kGivenWarps));
      heavy_piece[c] = x.hi > 0.0f;
      const Exact scan = scan_lanes(x, lane);
      end[c] = plus(total, scan);
      total = shuffled(end[c], 31);
    }
    if (total.hi > 0.0f || !(R.q || R.drop >= 0)) break;   // the same in the whole cluster
    R.q = nullptr;
    R.drop = -1;
  }
  cluster_sync_all();  // no CTA leaves while another may read its sums
  // ---- the crossing: one piece, the same choice in every warp --------------
  if (ok) {
    const Exact t = scaled(total, __ldg(a.sample_u + b));
    int winner = -1, heavy = -1;   // first piece that passes t; last one that weighs anything
#pragma unroll
    for (int c = 0; c < kMaxPieces / 32; ++c) {
      const unsigned pass = __ballot_sync(0xFFFFFFFFu, heavy_piece[c] && above(end[c], t));
      const unsigned some = __ballot_sync(0xFFFFFFFFu, heavy_piece[c]);
      if (winner < 0 && pass) winner = c * 32 + __ffs(pass) - 1;
      if (some) heavy = c * 32 + 31 - __clz(some);
    }
    if (winner < 0) winner = heavy;   // s >= 1, or a sum that is not finite
    if (total.hi > 0.0f && winner >= 0 && winner / kGivenWarps == rank) {
      // the CTA that owns it splits the piece over its warps once more, so that
      // the last look through single entries is short
      Exact before = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kMaxPieces / 32; ++c) {
        const Exact e = shuffled(end[c], (winner - 1) & 31);
        if (winner > 0 && (winner - 1) / 32 == c) before = e;
      }
      int p0 = min(a.V, winner * len), p1 = min(a.V, p0 + len), part_len = len;
      int pick, q0, q1;
      Exact pick_at;
      while (true) {
        part_len = ((part_len + kGivenWarps - 1) / kGivenWarps + 3) & ~3;
        q0 = min(p1, p0 + warp * part_len);
        q1 = min(p1, q0 + part_len);
        const Exact part = piece_sum<LONG>(R, q0, q1, lane);
        if (lane == 0) parts[warp] = part;
        __syncthreads();
        pick = -1;
        int some = -1;
        Exact at = before, some_at = before;
        pick_at = before;
#pragma unroll
        for (int w = 0; w < kGivenWarps; ++w) {
          const Exact y = parts[w], next = plus(at, y);
          if (y.hi > 0.0f) {
            some = w;
            some_at = at;
            if (pick < 0 && above(next, t)) {
              pick = w;
              pick_at = at;
            }
          }
          at = next;
        }
        if (pick < 0) {   // rounding at the piece's very end
          pick = some;
          pick_at = some_at;
        }
        if (!LONG || part_len <= kLook || pick < 0) break;   // the same in every warp
        p0 = min(p1, p0 + pick * part_len);
        p1 = min(p1, p0 + part_len);
        before = pick_at;
        __syncthreads();   // parts are read before the next round's
      }
      if (pick == warp) {
        const int token = piece_find(R, q0, q1, pick_at, t, lane);
        if (lane == 0) a.out_tokens[d0 + b + n] = token;
      }
    }
    if (rank == 0) {
      if (tid == 0) {
        a.out_nacc[b] = n;
        if (!(total.hi > 0.0f)) a.out_tokens[d0 + b + n] = 0;   // a row without weight
      }
      for (int i = n + 1 + tid; i <= gamma; i += kGivenThreads) a.out_tokens[d0 + b + i] = -1;
    }
  }
}

}  // namespace

int launch_given(const GivenArgs& a, int num_sms, cudaStream_t st) {
  // CTAs of a request: as many as give every warp a step of its row and as one wave
  // holds (4 CTAs of an SM are resident).  us with half, with these and with twice as many:
  // 64 requests of 151936 entries 24, 21, - (4, 8 CTAs); 128 40, 34, 35; 160 60, 44, 46; 256
  // 72, 59, 60; 304 of 128000 66, 55, 59.  Of more requests than a wave of single CTAs
  // takes, short rows lose by two of them (400 of 32000 24 and 26) and long ones would
  // gain (512 of 128000 95 and 91, 480 of 151936 108 and 102): one serves both.
  int C = kMaxCtas;
  while (C > 1 && (a.V < C * kGivenWarps * kStep || (int64_t)a.B * C > (int64_t)num_sms * 4)) C >>= 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * C);
  cfg.blockDim = dim3(kGivenThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool is_long = a.V > C * kGivenWarps * kChunk;
  return cudaLaunchKernelEx(&cfg, is_long ? given_kernel<true> : given_kernel<false>, a) == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace specdec
