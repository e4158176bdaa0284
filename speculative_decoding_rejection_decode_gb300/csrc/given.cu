// Verification of drafted chains from target probabilities and given random
// numbers.  Contract in include/specdec.h (specdec_rejection_sample_given).
//
// Only one target row (and, after a rejection, one draft row) of a request is
// read in full: the accept tests need single entries.  The extra token is the
// inverse of the cumulative weights, t = first v with C(v) > s C(V - 1), so the
// sums decide a whole number and are held to about 2^-48: every lane keeps a
// pair of floats (Knuth's two-sum gives each rounding error exactly), pairs
// meet in double precision.  A double addition per entry instead would be
// bound by the FP64 pipe, not by memory.
//
// A request is a cluster of C CTAs.  Each warp of the cluster sums a contiguous
// piece of the row; the piece sums meet in distributed shared memory (no
// workspace, no atomics, a fixed order); the CTA whose piece holds the crossing
// reads it again, from L2, first by warps and then entry by entry.
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

struct Pair {  // hi + lo, |lo| at most a few roundings of hi
  float hi, lo;
};

__device__ __forceinline__ void two_sum(Pair& s, float x) {
  const float t = __fadd_rn(s.hi, x);
  const float b = __fsub_rn(t, s.hi);
  const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x, b));
  s.hi = t;
  s.lo = __fadd_rn(s.lo, e);
}

// max(0, p - q) with the rounding error of the difference (0 where p <= q).
// Entries that are not above 0 (NaN among them) weigh nothing.
__device__ __forceinline__ void weigh(float p, float q, float& w, float& e) {
  const float d = __fsub_rn(p, q);
  const float b = __fsub_rn(d, p);
  const float r = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
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

__device__ __forceinline__ void weights4(const Rows& R, int v, const float* p, const float* q,
                                         float* w, float* e) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float qq = R.q ? q[k] : (v + k == R.drop ? 1.0f : 0.0f);
    weigh(p[k], qq, w[k], e[k]);
  }
}

// Sum of the weights of [v0, v1) (v0 a multiple of 4) over the warp.
__device__ __forceinline__ double piece_sum(const Rows& R, int v0, int v1, int lane) {
  Pair s = {0.0f, 0.0f};
  constexpr int U = 4;
  for (int base = v0; base < v1; base += U * kStep) {
    float p[U][4], q[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = base + u * kStep + lane * 4;
      if (v < v1) {
        load4(R.p, v, v1, R.vec, p[u]);
        if (R.q) load4(R.q, v, v1, R.vec, q[u]);
      } else {
        p[u][0] = p[u][1] = p[u][2] = p[u][3] = 0.0f;
        q[u][0] = q[u][1] = q[u][2] = q[u][3] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float w[4], e[4];
      weights4(R, base + u * kStep + lane * 4, p[u], q[u], w, e);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        two_sum(s, w[k]);
        s.lo = __fadd_rn(s.lo, e[k]);
      }
    }
  }
  double d = (double)s.hi + (double)s.lo;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
  return d;
}

// First v of [v0, v1) whose cumulative weight (after `before`) is above t;
// the last entry that weighs anything where rounding hides it.
__device__ __forceinline__ int piece_find(const Rows& R, int v0, int v1, double before, double t, int lane) {
  int last = v0;
  for (int base = v0; base < v1; base += kStep) {
    const int v = base + lane * 4;
    float p[4] = {}, q[4] = {}, w[4], e[4];
    if (v < v1) {
      load4(R.p, v, v1, R.vec, p);
      if (R.q) load4(R.q, v, v1, R.vec, q);
    }
    weights4(R, v, p, q, w, e);
    double c[4], sum = 0.0;
    int mine = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      sum += (double)w[k] + (double)e[k];
      c[k] = sum;
      if (w[k] > 0.0f) mine = v + k;
    }
    double scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
      if (lane >= o) scan += up;
    }
    const double at = before + (scan - sum);
    int hit = -1;
#pragma unroll
    for (int k = 3; k >= 0; --k)
      if (w[k] > 0.0f && at + c[k] > t) hit = v + k;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, hit >= 0);
    if (who) return __shfl_sync(0xFFFFFFFFu, hit, __ffs(who) - 1);
    const unsigned some = __ballot_sync(0xFFFFFFFFu, mine >= 0);
    if (some) last = __shfl_sync(0xFFFFFFFFu, mine, 31 - __clz(some));
    before += __shfl_sync(0xFFFFFFFFu, scan, 31);
  }
  return last;
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double d;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(d) : "r"(addr) : "memory");
  return d;
}

__global__ void __launch_bounds__(kGivenThreads) given_kernel(const GivenArgs a) {
  __shared__ double sums[2][kGivenWarps], parts[kGivenWarps];
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
  double total = 0.0, x[kMaxPieces / 32], end[kMaxPieces / 32];
  for (int round = 0; round < 2; ++round) {
    const double own_sum = ok ? piece_sum(R, v0, v1, lane) : 0.0;
    if (lane == 0) sums[round][warp] = own_sum;
    cluster_sync_all();
    // the same order in every warp: lane l holds pieces l and l + 32
    total = 0.0;
#pragma unroll
    for (int c = 0; c < kMaxPieces / 32; ++c) {
      const int k = c * 32 + lane;
      x[c] = 0.0;
      if (k < pieces)
        x[c] = ld_cluster_f64(mapa(smem_addr(&sums[round][k % kGivenWarps]), k / kGivenWarps));
      double scan = x[c];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += up;
      }
      end[c] = total + scan;
      total += __shfl_sync(0xFFFFFFFFu, scan, 31);
    }
    if (total > 0.0 || !(R.q || R.drop >= 0)) break;   // the same in the whole cluster
    R.q = nullptr;
    R.drop = -1;
  }
  cluster_sync_all();  // no CTA leaves while another may read its sums
  // ---- the crossing: one piece, the same choice in every warp --------------
  if (ok) {
    const double t = (double)__ldg(a.sample_u + b) * total;
    int winner = -1, heavy = -1;   // first piece that passes t; last one that weighs anything
    double before = 0.0;
#pragma unroll
    for (int c = 0; c < kMaxPieces / 32; ++c) {
      const unsigned pass = __ballot_sync(0xFFFFFFFFu, x[c] > 0.0 && t < end[c]);
      const unsigned some = __ballot_sync(0xFFFFFFFFu, x[c] > 0.0);
      if (winner < 0 && pass) winner = c * 32 + __ffs(pass) - 1;
      if (some) heavy = c * 32 + 31 - __clz(some);
    }
    if (winner < 0) winner = heavy;   // s >= 1, or a sum that is not finite
    if (total > 0.0 && winner >= 0 && winner / kGivenWarps == rank) {
      // the CTA that owns it splits the piece over its warps once more, so that
      // the last look through single entries is short
#pragma unroll
      for (int c = 0; c < kMaxPieces / 32; ++c) {
        const double e = __shfl_sync(0xFFFFFFFFu, end[c], (winner - 1) & 31);
        if (winner > 0 && (winner - 1) / 32 == c) before = e;
      }
      const int p0 = min(a.V, winner * len), p1 = min(a.V, p0 + len);
      const int len2 = ((len + kGivenWarps - 1) / kGivenWarps + 3) & ~3;
      const int q0 = min(p1, p0 + warp * len2), q1 = min(p1, q0 + len2);
      const double part = piece_sum(R, q0, q1, lane);
      if (lane == 0) parts[warp] = part;
      __syncthreads();
      int pick = -1, some = -1;
      double at = before, pick_at = before, some_at = before;
#pragma unroll
      for (int w = 0; w < kGivenWarps; ++w) {
        const double y = parts[w];
        if (y > 0.0) {
          some = w;
          some_at = at;
          if (pick < 0 && t < at + y) {
            pick = w;
            pick_at = at;
          }
        }
        at += y;
      }
      if (pick < 0) {   // rounding at the piece's very end
        pick = some;
        pick_at = some_at;
      }
      if (pick == warp) {
        const int token = piece_find(R, q0, q1, pick_at, t, lane);
        if (lane == 0) a.out_tokens[d0 + b + n] = token;
      }
    }
    if (rank == 0) {
      if (tid == 0) {
        a.out_nacc[b] = n;
        if (!(total > 0.0)) a.out_tokens[d0 + b + n] = 0;   // a row without weight
      }
      for (int i = n + 1 + tid; i <= gamma; i += kGivenThreads) a.out_tokens[d0 + b + i] = -1;
    }
  }
}

}  // namespace

int launch_given(const GivenArgs& a, int num_sms, cudaStream_t st) {
  // CTAs of a request: as many as give every warp a step of its row and as one wave
  // holds (4 CTAs of an SM are resident).  256 requests of 151936 entries: 2 CTAs
  // each took 81 us, 1 112, 4 85, 8 94; 8 requests of 32000: 8 CTAs 11 us, 4 12, 1 21.
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
  return cudaLaunchKernelEx(&cfg, given_kernel, a) == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace specdec
