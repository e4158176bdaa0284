// What the tensor-core attention kernels share: tcgen05 and TMA instructions, operand
// layouts, bounded waits, the segments of a CTA's range (attention_tile.cuh,
// cross_wide.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention.cuh"

namespace specdec {
namespace {

constexpr int kR = 128, kTK = 128;   // rows and keys of a product's tile

// ---- tcgen05 -------------------------------------------------------------------
// Issued by the one thread that elect.sync names, in a branch of its own: eight products
// with a factor in tensor memory are handed over in 63 clocks then, where a predicate on
// the lane takes 483 (66 each, whatever their size: what one of 128 x 128 x 16 runs for) and
// keeps the tensor cores waiting at every pause.  A converged warp calls; the thread is the
// same one every time, so that a commit covers the products before it.
__device__ __forceinline__ bool tc_elect() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// d (+)= A B, both in shared memory
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// the same for e4m3 factors, 32 of the summed dimension
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// d (+)= A B, A in tensor memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}

// Neighbouring columns of this thread's lane.  The wait stands in the same
// statement, so that no use of the values can move before it.
__device__ __forceinline__ void tc_ld32(uint32_t addr, float* x) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]),"=r"(r[1]),"=r"(r[2]),"=r"(r[3]),"=r"(r[4]),"=r"(r[5]),"=r"(r[6]),"=r"(r[7]),"=r"(r[8]),"=r"(r[9]),"=r"(r[10]),"=r"(r[11]),"=r"(r[12]),"=r"(r[13]),"=r"(r[14]),"=r"(r[15]),"=r"(r[16]),"=r"(r[17]),"=r"(r[18]),"=r"(r[19]),"=r"(r[20]),"=r"(r[21]),"=r"(r[22]),"=r"(r[23]),"=r"(r[24]),"=r"(r[25]),"=r"(r[26]),"=r"(r[27]),"=r"(r[28]),"=r"(r[29]),"=r"(r[30]),"=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptor: swizzled rows of LINE = 128 (or 64) bytes in
// groups of 8.  `lead`: bytes between 64-element chunks where the contiguous
// dimension is not the one summed over (V).
template <int LINE = 128>
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  const uint32_t lo = ((addr >> 4) & 0x3FFFu) | ((lead >> 4) << 16);
  const uint32_t hi = (8u * LINE >> 4) | (1u << 14) | ((LINE == 128 ? 2u : 4u) << 29);
  return ((uint64_t)hi << 32) | lo;
}

// Instruction descriptors: f32 accumulators, 128 x n; 16-bit or e4m3 factors.
template <typename E>
__device__ __forceinline__ constexpr uint32_t product(int n, bool b_rows_summed) {
  const uint32_t t = std::is_same<E, __half>::value ? 0u : 1u;
  return (1u << 4) | (t << 7) | (t << 10) | (b_rows_summed ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kR >> 4) << 24);
}
__device__ __forceinline__ constexpr uint32_t product_e4m3(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kR >> 4) << 24);
}

// Byte offset of 16-byte chunk c (of the row's 16-bit values) of row r of an
// operand tile: [64-value half][row][128 bytes], chunks spread by the row.
__device__ __forceinline__ uint32_t op_chunk(int r, int c) {
  return (uint32_t)((c >> 3) * (kTK * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The same for a tile of 8-bit rows of D bytes.
template <int D>
__device__ __forceinline__ uint32_t byte_chunk(int r, int c) {
  return (uint32_t)(r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
// Arrives on `bar` once every copy that this thread has issued has landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// A box of rows `row`, ... from column x of the map's array; completes on `bar`.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(row), "r"(one)
      : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 32 bytes in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 16 neighbouring floats in pairs, their loads under way together.
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t* f) {
  asm volatile(
      "ld.shared.v2.u64 {%0,%1}, [%8];\n\tld.shared.v2.u64 {%2,%3}, [%8+16];\n\t"
      "ld.shared.v2.u64 {%4,%5}, [%8+32];\n\tld.shared.v2.u64 {%6,%7}, [%8+48];"
      : "=l"(f[0]), "=l"(f[1]), "=l"(f[2]), "=l"(f[3]), "=l"(f[4]), "=l"(f[5]), "=l"(f[6]), "=l"(f[7])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A wait that gives up: the role goes on without waiting (its loops are finite
// and its addresses do not depend on data), and the call reports the timeout.  A
// try on a phase that does not complete returns after 4.0 us on this GPU (measured: 2048 tries
// of 1, 32 and 128 threads, 4.2 us at most; the same with a time hint of 0.1 or 1 us, which
// therefore is not given), so that 2^20 of them end after 4.3 seconds; the other roles'
// waits end within 256 of theirs, a millisecond.
// (Kept this small because it stands in many places: with a clock read in each,
// the kernel's code passed the instruction cache.)
__device__ __forceinline__ void wait_or_give_up(int& dead, uint32_t bar, uint32_t parity) {
  for (int i = 0; i < (1 << 20); ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return;
    if ((i & 255) == 255 && *reinterpret_cast<volatile int*>(&dead)) return;
  }
  *reinterpret_cast<volatile int*>(&dead) = 1;
}

// The segments of this CTA's range; every role steps through them by itself, on a
// copy in shared memory (registers are short).
struct Segments {
  int64_t base;      // units before request b
  int64_t end;
  Request q;
  int b, h, rt, t0, t1, rows;
  int u;             // next unit, from base
  bool whole, more;
};

template <int R>   // rows of a tile
__device__ __forceinline__ void next_segment(Segments* s, const PlanArgs c) {
  s->more = false;
  do {
    if (s->base + s->u >= s->end) return;
    uint32_t ignored = 0;
    while (s->u >= (int)s->q.units) {
      s->base += s->q.units;
      s->u -= (int)s->q.units;
      if (++s->b >= c.B) return;   // lengths that changed under the call
      s->q = attend_request(c, s->b, R, kTK, ignored);
    }
    const int tiles = c.whole ? 1 : s->q.tiles, rts = s->q.rts, u = s->u;
    const int item = (int)((unsigned)u / (unsigned)(tiles + c.item_cost)), at = u - item * (tiles + c.item_cost);
    s->t0 = max(at - c.item_cost, 0);
    s->t1 = (int)min((int64_t)tiles, at - c.item_cost + (s->end - s->base - u));
    s->h = (int)((unsigned)item / (unsigned)rts);
    s->rt = item - s->h * rts;
    s->u = u + tiles + c.item_cost - at;
  } while (s->t1 <= s->t0);          // a range may end before an item's first tile
  if (c.whole) s->t1 = s->q.tiles;
  s->whole = s->t0 == 0 && s->t1 == s->q.tiles;
  s->rows = min(R, s->q.n * c.group - s->rt * R);
  s->more = true;
}

// Leaves a segment's item to the join if it begins here and goes on.
__device__ __forceinline__ void leave_open(OpenItem* open, const Segments& s, int64_t units, int G, int group) {
  if (s.whole || s.t0 > 0) return;
  open[blockIdx.x] = {s.q.first, s.base + s.u, units, s.q.n * group, s.h, s.rt, (int)min((int64_t)G, units)};
}

inline decltype(&cuTensorMapEncodeTiled) tensor_map_encoder() {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult got;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &got) != cudaSuccess ||
        got != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  return encode;
}

// The array of cache rows as TMA sees it: [rows, D] with boxes of `box` rows and
// 128 (8-bit: D) bytes, swizzled.  Encoded for every call: nothing is kept by an
// address.
inline bool encode_rows(CUtensorMap* map, const void* base, int64_t rows, int D, int box, bool fp8) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(D * (fp8 ? 1 : 2))};
  const cuuint32_t boxes[2] = {(cuuint32_t)(fp8 ? D : 64), (cuuint32_t)box}, steps[2] = {1, 1};
  return encode(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base),
                dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                fp8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace specdec
