// cross_wide_kernel: cross attention of many rows per request over 16-bit states, on the
// tensor cores (tcgen05, accumulators and weights in tensor memory).  Contract in
// include/specdec.h (specdec_cross_attention).
//
// A unit is 256 rows x 128 keys: two tiles of 128 rows meet every tile of keys and values
// that is fetched (one of 128 rows alone would ask L2 for more than it gives).  Per SM one
// CTA:
//   softmax (2 groups   group w has the rows of tile w, one a thread, so that nothing of a
//   of 4 warps)         row crosses threads: 32 scores at a time, fetched while the 32
//                       before are worked on;
//   products (1 warp)   ... P_0 V, S_0 of the next keys, P_1 V, S_1 of the next ...: while one
//                       group works on its scores, the other's products run (a warp for
//                       each group brought both into step, and the products stood still
//                       while both worked: 4000 clocks a unit);
//   loader (1 warp)     looks up the pages and brings keys and values by TMA boxes of 8 to 128
//                       rows of a page, and the next item's queries as soon as the last
//                       scores of this one are done;
//   finisher (1 warp)   takes out of a tile of values what no row may see (slots that are
//                       masked, missing or behind the last).
// Tensor memory: S_0, S_1 (P_w lies over S_w), O_0, O_1: 4 x 128 columns.
//
// Measured (32 query and 8 kv heads of 128, bf16): 8 requests of 1536 rows over 2816 states
// 566 GFLOP in 410 to 430 us = 1.3 PFLOP/s, the tensor pipe busy for 57 % of it; of 1000 to
// 2048 rows over 1500 to 4096 states 1.25.  Bound by a group's scores, exponentials and
// weights in turn with its products; neither unit is full.
#include "attention_tc.cuh"

namespace specdec {
namespace {

constexpr int kWideR = kWideRows;
constexpr int kGroup = 128;                          // threads of a softmax group, rows of its tile
constexpr int kProducts = 8, kLoad = 9, kFinish = 10;   // warps
constexpr int kWideThreads = 12 * 32;
constexpr int kFacts = 8;                            // tiles whose key facts are held

template <int D>
struct WideLayout {
  static constexpr int TB = kR * D * 2;              // an operand tile: 128 rows
  static constexpr int KS = D == 128 ? 2 : 4;        // tiles of keys and of values in flight
  static constexpr int VS = D == 128 ? 3 : 4;
  static constexpr int Q = 0;                        // [2]
  static constexpr int K = Q + 2 * TB;
  static constexpr int V = K + KS * TB;
  static constexpr int BYTES = V + VS * TB + 1024;   // and room to align
};

struct alignas(16) WideShared {   // live is read 16 bytes at a time
  uint64_t k_full[4], k_empty[4];
  uint64_t v_raw[4], v_full[4], v_empty[4];   // landed; what no row may see taken out; read
  uint64_t fact[kFacts];
  uint64_t s_full[2], p_full[2];              // scores; weights
  uint64_t q_full[2], q_empty, o_full[2];
  alignas(16) uint32_t live[kFacts][4];       // keys of a tile that rows see
  uint32_t tmem;
  int dead;                                   // a wait ran out
};

// Two 16-bit weights times `by`, rounded to 16 bits as well.
__device__ __forceinline__ uint32_t halves(uint32_t w, float by, __half) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(by));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t halves(uint32_t w, float by, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(by));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 32 neighbouring columns of this thread's lane, under way until tc_arrived.
__device__ __forceinline__ void tc_fetch32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]),"=r"(r[1]),"=r"(r[2]),"=r"(r[3]),"=r"(r[4]),"=r"(r[5]),"=r"(r[6]),"=r"(r[7]),"=r"(r[8]),"=r"(r[9]),"=r"(r[10]),"=r"(r[11]),"=r"(r[12]),"=r"(r[13]),"=r"(r[14]),"=r"(r[15]),"=r"(r[16]),"=r"(r[17]),"=r"(r[18]),"=r"(r[19]),"=r"(r[20]),"=r"(r[21]),"=r"(r[22]),"=r"(r[23]),"=r"(r[24]),"=r"(r[25]),"=r"(r[26]),"=r"(r[27]),"=r"(r[28]),"=r"(r[29]),"=r"(r[30]),"=r"(r[31])
      : "r"(addr));
}
// Every fetch has arrived; the values pass through, so that no use moves before.
__device__ __forceinline__ void tc_arrived(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]),"+r"(r[1]),"+r"(r[2]),"+r"(r[3]),"+r"(r[4]),"+r"(r[5]),"+r"(r[6]),"+r"(r[7]),"+r"(r[8]),"+r"(r[9]),"+r"(r[10]),"+r"(r[11]),"+r"(r[12]),"+r"(r[13]),"+r"(r[14]),"+r"(r[15]),"+r"(r[16]),"+r"(r[17]),"+r"(r[18]),"+r"(r[19]),"+r"(r[20]),"+r"(r[21]),"+r"(r[22]),"+r"(r[23]),"+r"(r[24]),"+r"(r[25]),"+r"(r[26]),"+r"(r[27]),"+r"(r[28]),"+r"(r[29]),"+r"(r[30]),"+r"(r[31]));
}

// What has been summed of a row so far times `fix`, a power of two (nearly, see below; weights
// take it rounded to 16 bits, to the power of two): the tile's weights that have been stored
// (`parts` x 32) and, where there is one, O_w.  Out of line: rare.
template <typename T, int D>
__device__ __noinline__ void rescale(uint32_t ts, uint32_t to, int parts, bool summed, float fix) {
  tc_wait_st();   // what is read back here has been stored
#pragma unroll 1
  for (int p = 0; p < parts; ++p) {
    uint32_t w16[16];
    tc_ld16(ts + p * 16, w16);
#pragma unroll
    for (int k = 0; k < 16; ++k) w16[k] = halves(w16[k], fix, T());
    tc_st16(ts + p * 16, w16);
  }
#pragma unroll 1
  for (int p = 0; summed && p < D / 16; ++p) {
    uint32_t o[16];
    tc_ld16(to + p * 16, o);
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fix);
    tc_st16(to + p * 16, o);
  }
}

// The reference of a row whose maximum has left the old one (-inf: none) behind.
__device__ __noinline__ float follow(float m, float most) { return m == -INFINITY ? most : m + ceilf(most - m); }

// A tile's scores of this thread's row become weights 2^(e - m), rounded to 16 bits for the
// product with V (half a step each at most) and summed unrounded, 32 at a time; the
// maximum of the next 32 is found beside the exponentials of these.  The reference m, the
// first maximum (so that a row that sees one state gets its values as they are), follows the
// maximum by whole numbers and only where that has passed it by kLazy: what has been summed
// is then multiplied by 2^(m - m'), a power of two but for |m'| 2^-24 (the rounding of m', as
// much as scores of that size are off by themselves).  (Handing on the first 96 keys'
// weights before the last 32 gained nothing.)
template <typename T, int D, bool MASKED>
__device__ __forceinline__ void tile_weights(uint32_t ts, uint32_t to, uint4 live, float rowf, bool summed,
                                             float& m, float& l, uint64_t* sum) {
  // f16 ends at 2^16; bf16, 8, 9 and 16: 456, 434 and 417 us, 8 requests of 1000 to 2048 rows
  // over 1500 to 4096 states.  bf16 weights end at 1, so that sums pass no further than the sum
  // of the values' magnitudes.
  constexpr float kLazy = std::is_same<T, __half>::value ? 9.0f : 16.0f;
  constexpr float kHead = std::is_same<T, __half>::value ? 6.0f : -kLazy;   // f16 weights keep their bits
  const uint64_t rowf2 = pair(rowf, rowf);
  uint32_t s[2][32];
  auto most_of = [&](uint32_t* x, uint32_t see) {
    if constexpr (MASKED) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (!((see >> k) & 1u)) x[k] = 0xFF800000u;
    }
    float q[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) q[z] = fmaxf(__uint_as_float(x[2 * z]), __uint_as_float(x[2 * z + 1]));
#pragma unroll
    for (int k = 8; k < 32; k += 8)
#pragma unroll
      for (int z = 0; z < 4; ++z) q[z] = max3(q[z], __uint_as_float(x[k + 2 * z]), __uint_as_float(x[k + 2 * z + 1]));
    return fmaxf(max3(q[0], q[1], q[2]), q[3]);
  };
  auto refer = [&](float mx, int parts) {
    const float most = mx == -INFINITY ? mx : mx * rowf;
    const bool move = most > m + kLazy || (m == -INFINITY && most != -INFINITY);
    if (__any_sync(0xFFFFFFFFu, move)) {
      const float to_m = move ? follow(m, most) : m;
      const float fix = move ? ex2(m - to_m) : 1.0f;
      m = to_m;
      l *= fix;
      const uint64_t fix2 = pair(fix, fix);
      sum[0] = mul2(sum[0], fix2);
      sum[1] = mul2(sum[1], fix2);
      if (parts > 0 || summed) rescale<T, D>(ts, to, parts, summed, fix);
    }
  };
  tc_fetch32(ts, s[0]);
  tc_fetch32(ts + 32, s[1]);
  tc_arrived(s[0]);
  refer(most_of(s[0], live.x), 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t *x = s[i & 1], *y = s[(i & 1) ^ 1];
    float mx = -INFINITY;
    if (i < 3) {
      tc_arrived(y);
      mx = most_of(y, i == 0 ? live.y : i == 1 ? live.z : live.w);
    }
    const float add = kHead - (m == -INFINITY ? 0.0f : m);
    const uint64_t add_2 = pair(add, add);
    uint32_t p[16];
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      float e0, e1;
      unpair(fma2(pair(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), rowf2, add_2), e0, e1);
      e0 = ex2(e0);
      e1 = ex2(e1);
      sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pair(e0, e1));
      p[k / 2] = pack2(e0, e1, T());
    }
    if (i < 2) tc_fetch32(ts + (i + 2) * 32, x);
    tc_st16(ts + i * 16, p);
    if (i < 3) refer(mx, i + 1);
  }
}

// A box of whole nodes' heads from (x, head, node) of the queries; completes on `bar`.
__device__ __forceinline__ void box3_load(uint32_t dst, const CUtensorMap* map, int x, int head, int node, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(head), "r"(node)
      : "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(kWideThreads, 1)
    cross_wide_kernel(const AttendArgs a, const int box, const bool qbox, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using L = WideLayout<D>;
  constexpr int CH = D / 8;                      // 16-byte chunks of an operand row
  extern __shared__ char smem_raw[];
  __shared__ ScanShared scan;
  __shared__ WideShared sh;
  // segments of the products, the loader, the finisher, and two of each softmax group
  __shared__ Segments segs[7];
  char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base_s = smem_addr(smem);
  const CacheArgs& c = a.c;
  const int G = gridDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.q_heads / c.geo.kv_heads;
  const PlanArgs plan(a);
  uint32_t why = 0;
  int64_t u0 = 0;
  find_unit<kWideThreads>(plan, kWideR, kTK,
                          [&](int64_t units) {
                            const int ranges = (int)min((int64_t)G, units);
                            u0 = (int)blockIdx.x < ranges ? range_begin(units, ranges, blockIdx.x) : units;
                            return u0;
                          },
                          scan, why);
  if (blockIdx.x == 0 && why) atomicOr(c.err, why);
  if (tid == 0 && !a.whole) Partials<kWideR, D>(a.workspace, G).open[blockIdx.x].ranges = 0;
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t units = scan.total;
  const int ranges = (int)min((int64_t)G, units);
  if ((int)blockIdx.x >= ranges || scan.b < 0) return;
  if (tid == 0) {
    for (int i = 0; i < L::KS; ++i) {
      mbar_init(smem_addr(&sh.k_full[i]), 1);
      mbar_init(smem_addr(&sh.k_empty[i]), 1);
    }
    for (int i = 0; i < L::VS; ++i) {
      mbar_init(smem_addr(&sh.v_raw[i]), 1);
      mbar_init(smem_addr(&sh.v_full[i]), 1);
      mbar_init(smem_addr(&sh.v_empty[i]), 1);
    }
    for (int i = 0; i < kFacts; ++i) mbar_init(smem_addr(&sh.fact[i]), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_addr(&sh.s_full[w]), 1);
      mbar_init(smem_addr(&sh.p_full[w]), 4);
      mbar_init(smem_addr(&sh.q_full[w]), qbox ? 1 : 4);
      mbar_init(smem_addr(&sh.o_full[w]), 1);
    }
    mbar_init(smem_addr(&sh.q_empty), 1);
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == kProducts) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "n"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sh.tmem;
  const int64_t uend = range_begin(units, ranges, blockIdx.x + 1);
  if (tid < 7) {
    uint32_t ignored = 0;
    Segments& s = segs[tid];
    s.end = uend;
    s.b = scan.b;
    s.base = scan.before;
    s.u = (int)(u0 - scan.before);
    s.q = attend_request(plan, scan.b, kWideR, kTK, ignored);
    next_segment<kWideR>(&s, plan);
  }
  __syncthreads();
  uint32_t bad = 0;
  auto wait_use = [&](uint64_t* bars, int slots, int n) {       // use n of a ring's slot is complete
    wait_or_give_up(sh.dead, smem_addr(&bars[n % slots]), (uint32_t)(n / slots) & 1u);
  };
  auto wait_free = [&](uint64_t* bars, int slots, int n) {      // the slot's use n - slots is complete
    wait_or_give_up(sh.dead, smem_addr(&bars[n % slots]), ((uint32_t)(n / slots) & 1u) ^ 1u);
  };
  if (warp == kProducts) {
    // ---- products ---------------------------------------------------------------
    Segments& seg = segs[0];
    auto scores = [&](int w, int slot) {         // the elected thread's
      const uint64_t qd = operand(base_s + L::Q + w * L::TB, 16), kd = operand(base_s + L::K + slot * L::TB, 16);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint32_t off = (uint32_t)((s >> 2) * (kTK * 128) + (s & 3) * 32) >> 4;
        tc_mma_ss(tm + w * 128, qd + off, kd + off, product<T>(kTK, false), s > 0);
      }
      tc_commit(smem_addr(&sh.s_full[w]));
    };
    int ks = 0, vs = 0;                          // slots of the next tiles of keys and values, and their phases
    uint32_t kp = 0, vp = 0, used = 0, begun = 0;   // bit w: phase of group w's weights, of its queries
    while (seg.more) {
      const int n = seg.t1 - seg.t0, tiles = seg.rows > kR ? 2 : 1;
      wait_or_give_up(sh.dead, smem_addr(&sh.k_full[ks]), kp);
#pragma unroll 1
      for (int w = 0; w < tiles; ++w) {
        wait_or_give_up(sh.dead, smem_addr(&sh.q_full[w]), (begun >> w) & 1u);
        begun ^= 1u << w;
        tc_fence_after();
        if (tc_elect()) {
          scores(w, ks);
          if (w + 1 == tiles) {
            tc_commit(smem_addr(&sh.k_empty[ks]));
            if (n == 1) tc_commit(smem_addr(&sh.q_empty));
          }
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if (++ks == L::KS) {
          ks = 0;
          kp ^= 1u;
        }
        wait_or_give_up(sh.dead, smem_addr(&sh.v_full[vs]), vp);
        if (j + 1 < n) wait_or_give_up(sh.dead, smem_addr(&sh.k_full[ks]), kp);
#pragma unroll 1
        for (int w = 0; w < tiles; ++w) {
          const uint32_t phase = (used >> w) & 1u;
          used ^= 1u << w;
          const uint64_t vd = operand(base_s + L::V + vs * L::TB, kTK * 128);
          wait_or_give_up(sh.dead, smem_addr(&sh.p_full[w]), phase);
          tc_fence_after();
          if (tc_elect()) {
#pragma unroll
            for (int s = 0; s < 8; ++s)
              tc_mma_ts(tm + 256 + w * 128, tm + w * 128 + s * 8, vd + (uint32_t)(s * 2048 >> 4), product<T>(D, true), s > 0 || j > 0);
            if (j + 1 < n) scores(w, ks);
            else tc_commit(smem_addr(&sh.o_full[w]));
            if (w + 1 == tiles) {
              tc_commit(smem_addr(&sh.v_empty[vs]));
              if (j + 1 < n) tc_commit(smem_addr(&sh.k_empty[ks]));
              if (j + 2 == n) tc_commit(smem_addr(&sh.q_empty));   // the segment's last scores
            }
          }
          __syncwarp();
        }
        if (++vs == L::VS) {
          vs = 0;
          vp ^= 1u;
        }
      }
      if (lane == 0) next_segment<kWideR>(&seg, plan);
      __syncwarp();
    }
  } else if (warp == kLoad) {
    // ---- loader -----------------------------------------------------------------
    // A box lies in one page: it is fetched if its first key lives, and what it brings of
    // slots behind the last key, or of masked ones, is hidden (keys) or taken out (values).
    // A lane looks up one box; 32 of them serve `batch` tiles.  (One tile's look-ups at a
    // time, and its boxes one after the other from one lane, took longer than the products:
    // 4700 clocks a unit.)
    Segments& seg = segs[1];
    constexpr int HALVES = D / 64;               // boxes of 64 values of a row
    const uint32_t page_size = (uint32_t)c.geo.page_size;
    const int shift = __ffs(box) - 1, boxes = kTK >> shift, batch = 32 / boxes;
    uint32_t begun = 0;                          // segments so far
    int n = 0;                                   // tiles so far
    while (seg.more) {
      const int t0 = seg.t0, t1 = seg.t1, h = seg.h;
      const uint32_t len = (uint32_t)seg.q.len;
      const int32_t* pages = c.table + seg.b * c.geo.table_stride;
      const uint8_t* mask = a.mask ? a.mask + seg.b * a.mask_stride : nullptr;
      int row = -1;                              // cache row of the first key of this lane's box
      for (int t = t0, p = batch; t < t1; ++t, ++n) {
        if (p == batch) {
          p = 0;
          const uint32_t key = (uint32_t)t * kTK + ((uint32_t)lane << shift), page = key / page_size;
          row = -1;
          if (key < len && t + lane / boxes < t1) {
            const int id = __ldg(pages + page);
            if (id >= 0 && id < c.geo.num_pages) row = (id * c.geo.kv_heads + h) * (int)page_size + (int)(key - page * page_size);
          }
        }
        const unsigned every = boxes == 32 ? 0xFFFFFFFFu : (1u << boxes) - 1u;
        const unsigned held = (__ballot_sync(0xFFFFFFFFu, row >= 0) >> (p * boxes)) & every;   // of this tile
        const uint32_t first = (uint32_t)t * kTK;
        const int f = n % kFacts;
        // (slot n % 8 is free: the waits for tile n - 5's slots below have passed)
        if (held == every && first + kTK <= len && !mask) {
          if (lane < 4) sh.live[f][lane] = 0xFFFFFFFFu;
        } else {
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const uint32_t in = i * 32 + lane, s = first + in;
            const bool shown = s < len && (!mask || (s < a.mask_slots && __ldg(mask + s))), here = (held >> (in >> shift)) & 1u;
            if (shown && !here) bad |= SPECDEC_DEVERR_BAD_CACHE;   // (a masked slot needs no page)
            const uint32_t live = __ballot_sync(0xFFFFFFFFu, shown && here);
            if (lane == 0) sh.live[f][i] = live;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.fact[f]));
        const int mine = __shfl_sync(0xFFFFFFFFu, row, (p * boxes + lane / HALVES) & 31);
        const bool fetches = lane < boxes * HALVES && mine >= 0;
        const uint32_t to = (uint32_t)(lane % HALVES) * (kTK * 128) + ((uint32_t)(lane / HALVES) << shift) * 128;
        auto fetch = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar) {
          if (lane == 0) mbar_arrive_expect_tx(bar, (__popc(held) << shift) * D * 2);
          __syncwarp();
          if (fetches) box_load(dst + to, map, lane % HALVES * 64, mine, bar, 1u);
        };
        wait_free(sh.k_empty, L::KS, n);
        fetch(base_s + L::K + (n % L::KS) * L::TB, &kmap, smem_addr(&sh.k_full[n % L::KS]));
        // queries that come by boxes of whole nodes (the group divides 128), read behind the last row too
        if (qbox && t == t0) {
          if (begun) wait_or_give_up(sh.dead, smem_addr(&sh.q_empty), (begun - 1) & 1u);
          ++begun;
          const int tiles = seg.rows > kR ? 2 : 1, node = (int)(seg.q.first + (int64_t)seg.rt * (kWideR / group));
          if (lane < tiles) mbar_arrive_expect_tx(smem_addr(&sh.q_full[lane]), L::TB);
          __syncwarp();
          if (lane < tiles * HALVES) {
            const int w = lane / HALVES, half = lane % HALVES;
            box3_load(base_s + L::Q + w * L::TB + half * (kR * 128), &qmap, half * 64, h * group, node + w * (kR / group),
                      smem_addr(&sh.q_full[w]));
          }
        }
        wait_free(sh.v_empty, L::VS, n);
        fetch(base_s + L::V + (n % L::VS) * L::TB, &vmap, smem_addr(&sh.v_raw[n % L::VS]));
        ++p;
      }
      __syncwarp();
      if (lane == 0) next_segment<kWideR>(&seg, plan);
      __syncwarp();
    }
  } else if (warp == kFinish) {
    // ---- finisher -------------------------------------------------------------------
    Segments& seg = segs[2];
    for (int n = 0, t = seg.t0; seg.more; ++n) {
      const int f = n % kFacts;
      wait_use(sh.fact, kFacts, n);
      const uint4 live = *reinterpret_cast<const uint4*>(sh.live[f]);
      wait_use(sh.v_raw, L::VS, n);
      if ((live.x & live.y & live.z & live.w) != 0xFFFFFFFFu) {
        const uint32_t dst = base_s + L::V + (n % L::VS) * L::TB;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {              // 32 keys at a time, one a lane
          const uint32_t see = i == 0 ? live.x : i == 1 ? live.y : i == 2 ? live.z : live.w;
          if ((see >> lane) & 1u) continue;
#pragma unroll 4
          for (int ch = 0; ch < CH; ++ch) sts128(dst + op_chunk(i * 32 + lane, ch), make_uint4(0, 0, 0, 0));
        }
        fence_async_proxy();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.v_full[n % L::VS]));
      if (++t == seg.t1) {
        __syncwarp();
        if (lane == 0) {
          leave_open(Partials<kWideR, D>(a.workspace, G).open, seg, scan.total, G, group);
          next_segment<kWideR>(&seg, plan);
        }
        __syncwarp();
        t = seg.t0;
      }
    }
  } else if (warp < kProducts) {
    // ---- softmax ----------------------------------------------------------------
    const int w = warp >> 2, in = tid & (kGroup - 1);            // group; row of its tile = lane of tensor memory
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;           // first lane, in bits 16..
    const uint32_t ts = tm + lanes + w * 128, to = tm + lanes + 256 + w * 128;
    const Partials<kWideR, D> part(a.workspace, G);
    // positive: hidden keys are -inf times this; the scale's sign goes to q
    const float rowf = fmaxf(fabsf(a.scale_log2), 1.17549435e-38f);
    Segments *cur = &segs[3 + 2 * w], *ahead = &segs[4 + 2 * w];
    int done = 0, tile0 = 0;                                     // this group's tiles; all tiles before the segment
    uint32_t g = 0;                                              // this group's segments
    auto queries = [&](const Segments& s) {
      if (!qbox && s.rows > w * kR) {
#pragma unroll 16
        for (int x = in; x < kR * CH; x += kGroup) {
          const int r = x / CH, ch = x % CH, of = w * kR + r;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (of < s.rows) {
            const int gr = s.rt * kWideR + of;
            v = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (s.q.first + gr / group) * a.q_row +
                                                     (int64_t)(s.h * group + gr % group) * a.q_head + ch * 8));
          }
          if (a.scale_log2 < 0.0f) {
            v.x ^= 0x80008000u;
            v.y ^= 0x80008000u;
            v.z ^= 0x80008000u;
            v.w ^= 0x80008000u;
          }
          sts128(base_s + L::Q + w * L::TB + op_chunk(r, ch), v);
        }
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[w]));
      }
    };
    if (cur->more) queries(*cur);
    while (cur->more) {
      // the segment after this one, while this one's keys are met
      named_bar_sync(1 + w, kGroup);
      if (in == 0) {
        *ahead = *cur;
        next_segment<kWideR>(ahead, plan);
      }
      const int n = cur->t1 - cur->t0;
      const bool active = cur->rows > w * kR;
      float m = -INFINITY, l = 0.0f;             // reference and sum of this row
      if (active) {
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int f = (tile0 + j) % kFacts;
          wait_use(sh.fact, kFacts, tile0 + j);
          wait_or_give_up(sh.dead, smem_addr(&sh.s_full[w]), (uint32_t)done & 1u);
          ++done;
          tc_fence_after();
          const uint4 live = *reinterpret_cast<const uint4*>(sh.live[f]);
          uint64_t sum[2] = {0, 0};
          if ((live.x & live.y & live.z & live.w) == 0xFFFFFFFFu) tile_weights<T, D, false>(ts, to, live, rowf, j > 0, m, l, sum);
          else tile_weights<T, D, true>(ts, to, live, rowf, j > 0, m, l, sum);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[w]));
          float s0, s1;
          unpair(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
        }
      }
      tile0 += n;
      // every score of the segment is done: the next one's queries, then this one's results
      named_bar_sync(1 + w, kGroup);
      if (ahead->more) queries(*ahead);
      if (active) {
        const Segments& seg = *cur;
        wait_or_give_up(sh.dead, smem_addr(&sh.o_full[w]), g & 1u);
        ++g;
        tc_fence_after();
        const int of = w * kR + in, gr = seg.rt * kWideR + of;
        const bool live = of < seg.rows;
        const float inv = seg.whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (seg.t0 > 0 ? 0 : 1);
        const bool aligned = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        const int64_t at = (seg.q.first + gr / group) * a.q_heads + seg.h * group + gr % group;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float x[32];
          __syncwarp();
          tc_ld32(to + i * 32, x);
          if (!live) continue;
          // (a reference of -inf may also mean that what the row saw was no number: inv is NaN then)
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = (m == -INFINITY ? 0.0f : x[k]) * inv;
          // (a row's own lines: 32 bytes a store, half as many stores as of 16)
          if (seg.whole && aligned) {
            T* out = static_cast<T*>(a.out) + at * D + i * 32;
            uint32_t y[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = pack2(x[2 * k], x[2 * k + 1], T());
            store32(out, y);
            store32(out + 16, y + 8);
          } else if (seg.whole) {
            T* out = static_cast<T*>(a.out) + at * D + i * 32;
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              *reinterpret_cast<uint4*>(out + k) = make_uint4(pack2(x[k], x[k + 1], T()), pack2(x[k + 2], x[k + 3], T()),
                                                              pack2(x[k + 4], x[k + 5], T()), pack2(x[k + 6], x[k + 7], T()));
          } else {
            float* out = part.sums + (slot * kWideR + of) * D + i * 32;
#pragma unroll
            for (int k = 0; k < 32; k += 8) store32(out + k, reinterpret_cast<const uint32_t*>(x + k));
          }
        }
        if (live && !seg.whole) part.stats[slot * kWideR + of] = make_float2(m, l);
        tc_fence_before();                       // the sums are read before the next segment's lie over them
      }
      named_bar_sync(1 + w, kGroup);
      Segments* x = cur;
      cur = ahead;
      ahead = x;
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
  if (warp == kProducts)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(512));
}

// Queries [N, q_heads, D] in their strides, boxes of 64 values x the heads of a kv head x
// the nodes of a tile.  False where TMA has no such strides.
bool encode_queries(CUtensorMap* map, const AttendArgs& a, int D, int group) {
  const auto encode = tensor_map_encoder();
  const int64_t head = a.q_heads > 1 ? 2 * a.q_head : 2 * D, row = a.c.N > 1 ? 2 * a.q_row : 2 * D * a.q_heads;
  if (!encode || head <= 0 || row <= 0 || head >= ((int64_t)1 << 40) || row >= ((int64_t)1 << 40)) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.q_heads, (cuuint64_t)a.c.N};
  const cuuint64_t strides[2] = {(cuuint64_t)head, (cuuint64_t)row};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)group, (cuuint32_t)(kR / group)}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(a.q), dims, strides, boxes, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
int launch_wide(const AttendArgs& a, int box, int num_sms, cudaStream_t st) {
  auto kern = cross_wide_kernel<T, D>;
  constexpr int bytes = WideLayout<D>::BYTES;
  static std::atomic<uint64_t> done{0};
  if (!allow_shared(kern, bytes, done)) return SPECDEC_ERR_CUDA;
  CUtensorMap kmap = {}, vmap = {}, qmap = {};
  const int64_t rows = a.c.geo.num_pages * a.c.geo.kv_heads * a.c.geo.page_size;
  if (!encode_rows(&kmap, a.c.k, rows, D, box, false) || !encode_rows(&vmap, a.c.v, rows, D, box, false)) return SPECDEC_ERR_CUDA;
  // Queries by boxes where whole nodes fill a tile and nothing is to be done to them; else
  // the softmax groups bring them (17500 clocks an item, and nothing else going on, where
  // boxes are there when they are needed).
  const int group = a.q_heads / a.c.geo.kv_heads;
  const bool qbox = kR % group == 0 && a.scale_log2 >= 0.0f && encode_queries(&qmap, a, D, group);
  kern<<<num_sms, kWideThreads, bytes, st>>>(a, box, qbox, kmap, vmap, qmap);
  if (cudaGetLastError() != cudaSuccess) return SPECDEC_ERR_CUDA;
  return a.whole ? SPECDEC_OK : launch_join<T, kWideR, D>(a, num_sms, st);
}

}  // namespace

int64_t cross_wide_workspace(int head_dim, int num_sms) {
  return head_dim == 128 ? Partials<kWideR, 128>::bytes(num_sms) : Partials<kWideR, 64>::bytes(num_sms);
}

int launch_cross_wide(const AttendArgs& a, int dtype, int num_sms, cudaStream_t st) {
  // rows of a box: within one page, whole groups of 8 rows of the swizzle
  int box = 128;
  while (box > 8 && a.c.geo.page_size % box) box >>= 1;
  if (dtype == SPECDEC_BF16)
    return a.c.head_dim == 128 ? launch_wide<__nv_bfloat16, 128>(a, box, num_sms, st) : launch_wide<__nv_bfloat16, 64>(a, box, num_sms, st);
  return a.c.head_dim == 128 ? launch_wide<__half, 128>(a, box, num_sms, st) : launch_wide<__half, 64>(a, box, num_sms, st);
}

}  // namespace specdec
