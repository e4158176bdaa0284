// Index arithmetic of the paged key/value cache and of token trees: plain C++
// that the kernels and the host share, so that every bound can be checked
// without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SPECDEC_HD __host__ __device__ __forceinline__
#else
#define SPECDEC_HD inline
#endif

namespace specdec {

// Geometry of a cache: rows of head_dim values, [num_pages, kv_heads,
// page_size], and of the page table [B, max_pages] (rows table_stride apart).
struct PagedGeo {
  int64_t num_pages;
  int64_t table_stride;
  int32_t kv_heads;
  int32_t page_size;
  int32_t max_pages;
};

// Nodes of request b: the first one and their number.  A cu that decreases,
// starts below 0 or passes the N rows given is not a range (false).
SPECDEC_HD bool node_range(const int32_t* cu, int b, int64_t N, int64_t& first, int32_t& count) {
  const int64_t a = cu[b], z = cu[b + 1];
  if (a < 0 || z < a || z > N) return false;
  first = a;
  count = (int32_t)(z - a);
  return true;
}

// Request that owns row r (cu[b] <= r < cu[b + 1]), or -1: the largest b with
// cu[b] <= r by bisection, then a check, so that any cu ends the search.
SPECDEC_HD int request_of_row(const int32_t* cu, int B, int64_t r) {
  int lo = 0, hi = B;  // cu[lo] <= r is assumed of lo, r < cu[hi] of hi
  while (hi - lo > 1) {
    const int mid = lo + ((hi - lo) >> 1);
    if ((int64_t)cu[mid] <= r) lo = mid; else hi = mid;
  }
  return ((int64_t)cu[lo] <= r && r < (int64_t)cu[lo + 1]) ? lo : -1;
}

// Row of cache head 0 that holds `slot` of the request whose table row is
// `pages`; head h lies h * page_size rows further.  -1 for a slot or a page
// id outside the table or the cache: the caller skips the access.
SPECDEC_HD int64_t cache_row(const PagedGeo& g, const int32_t* pages, int64_t slot) {
  if (slot < 0 || slot > 0xFFFFFFFFll) return -1;  // lengths and nodes are 32-bit
  const uint32_t at = (uint32_t)slot / (uint32_t)g.page_size;
  if (at >= (uint32_t)g.max_pages) return -1;
  const int64_t page = pages[at];
  if (page < 0 || page >= g.num_pages) return -1;
  return page * g.kv_heads * g.page_size + ((uint32_t)slot - at * (uint32_t)g.page_size);
}

// Depth of node j below its request's node 0, from parents within the request
// (parents lie before their children, the root has -1); null parents are a
// chain.  -1 when the walk meets a parent that is no earlier node, or ends at
// a node other than 0.
SPECDEC_HD int node_depth(const int32_t* parent, int j) {
  if (!parent) return j;
  int depth = 0;
  while (j > 0) {
    const int up = parent[j];
    if (up < 0 || up >= j) return -1;
    j = up;
    ++depth;
  }
  return depth;
}

// The flattened attention work: request b has items(b) = kv_heads * row tiles,
// each of tiles(b) key tiles; the units of all requests, in that order, are
// split into G equal contiguous ranges.
SPECDEC_HD int64_t range_begin(int64_t units, int G, int i) {
  // units < 2^53 and G small: the quotient is taken apart so that nothing overflows
  return (units / G) * i + (units % G) * i / G;
}

// Range that owns unit u (range_begin(i) <= u < range_begin(i + 1)).
SPECDEC_HD int range_of(int64_t units, int G, int64_t u) {
  int i = (int)((double)u / (double)units * G);
  if (i >= G) i = G - 1;
  while (i > 0 && range_begin(units, G, i) > u) --i;
  while (i < G - 1 && range_begin(units, G, i + 1) <= u) ++i;
  return i;
}

}  // namespace specdec
