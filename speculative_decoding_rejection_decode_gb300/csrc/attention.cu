// Attention over the paged cache: which kernel serves a call (attention_warp.cuh for few
// rows per request, attention_tile.cuh for many), and its workspace.
#include "attention_warp.cuh"

namespace specdec {
namespace {

// Rows (nodes x heads that share a kv head) of an average request: what the
// host knows of the rows of a tile.
int64_t average_rows(int B, int64_t N, int kv_heads, int q_heads) {
  return (N + B - 1) / B * (q_heads / kv_heads);
}
// Up to these (a tile of the warp kernel) the warp kernel, above them the tile kernel.
// One context of 500 / 64 up to 8191 / 4 of 30000 / 200 up to 1500, 8 kv heads of 128,
// device us, warp and tile kernel:
//   4 rows  bf16 14.9 18.1 / 179 184 / 87 90 / 127 150, e4m3 14.8 18.9 / 179 208 / 81 81 / 152 197
//   12      bf16 16.8 18.8 / 183 185 / 92 92 / 144 151, e4m3 16.8 19.1 / 188 206 / 85 82 / 172 199
//   16      bf16 17.3 18.8 / 182 185 / 93 92 / 148 151, e4m3 16.9 19.4 / 192 207 / 86 82 / 177 199
//   20      bf16 17.0 18.9 / 340 189 / 165 94 / 255 153, e4m3 18.4 19.0 / 345 210 / 146 82 / 306 198
// The average decides: in a batch of one large request among many small ones, the
// large one takes a tile of 16 rows at a time.
constexpr int kWarpRows = 16;

// Which kernel serves a call.
enum class Kernel { kWarp, kTile, kWide };

constexpr int kTileRows = 128;   // rows of a tile of the tile kernel

// The wide kernel (cross_wide.cu) reads a key for 256 rows, and is bound by the products; the
// tile kernel divides a call's rows among more CTAs.  Tile and wide kernel, device us, 32
// query and 8 kv heads of 128, bf16 states (rows of a request and kv head):
//   1 request, 2816 states    128  29 29    160  27 31    256  29 36    512  31 37
//   8 of 2816                 128  46 50    160  53 54    384  70 74    512  84 79
//   64 of 1500                128 115 116   144 171 127   256 193 136   512 349 221
// The wide one takes over where the rows pass a tile and the tiles are more than one and a
// half for each SM.
Kernel kernel_of(bool cross, int cache_dtype, int page_size, int B, int64_t N, int kv_heads, int q_heads, int num_sms) {
  const int64_t avg = average_rows(B, N, kv_heads, q_heads);
  if (avg <= kWarpRows) return Kernel::kWarp;
  const int64_t tiles = (int64_t)B * kv_heads * ((avg + kTileRows - 1) / kTileRows);
  return cross && cache_dtype != SPECDEC_E4M3 && page_size % 8 == 0 && avg > kTileRows && 2 * tiles > 3 * (int64_t)num_sms
             ? Kernel::kWide : Kernel::kTile;
}

int rows_of(Kernel k) { return k == Kernel::kWarp ? kRowsTile : k == Kernel::kTile ? kTileRows : kWideRows; }

}  // namespace

int64_t attend_workspace_bytes(bool cross, int cache_dtype, int page_size, int B, int64_t N, int kv_heads, int q_heads,
                               int head_dim, int64_t capacity, int num_sms) {
  const Kernel k = kernel_of(cross, cache_dtype, page_size, B, N, kv_heads, q_heads, num_sms);
  if (whole_items(B, N, kv_heads, q_heads, capacity, rows_of(k), num_sms)) return 0;
  if (k == Kernel::kWide) return cross_wide_workspace(head_dim, num_sms);
  if (k == Kernel::kTile) return attend_tile_workspace(head_dim, num_sms);
  return head_dim == 128 ? Partials<kRowsTile, 128>::bytes(num_sms) : Partials<kRowsTile, 64>::bytes(num_sms);
}

int launch_attend(const AttendArgs& args, int cache_dtype, int dtype, int num_sms, cudaStream_t st) {
  if (args.c.N == 0) return SPECDEC_OK;
  AttendArgs a = args;
  const CacheArgs& c = a.c;
  const Kernel k = kernel_of(a.cross, cache_dtype, c.geo.page_size, c.B, c.N, c.geo.kv_heads, a.q_heads, num_sms);
  a.whole = whole_items(c.B, c.N, c.geo.kv_heads, a.q_heads, (int64_t)c.geo.max_pages * c.geo.page_size, rows_of(k), num_sms);
  const bool fp8 = cache_dtype == SPECDEC_E4M3;
  const bool brief = !a.cross && (int64_t)c.geo.max_pages * c.geo.page_size <= kShortSlots;
  a.item_cost = k == Kernel::kWide ? kItemCostWide : !fp8 ? kItemCost : k == Kernel::kWarp ? kItemCostWarp8
              : brief ? kItemCostTile8Short : kItemCostTile8;
  if (k == Kernel::kWide) return launch_cross_wide(a, dtype, num_sms, st);
  if (k == Kernel::kTile) return a.cross ? launch_cross_tile(a, cache_dtype, dtype, num_sms, st) : launch_attend_tile(a, cache_dtype, dtype, num_sms, st);
  return a.cross ? launch_cross_warp(a, cache_dtype, dtype, num_sms, st) : launch_warp_types<false>(a, cache_dtype, dtype, num_sms, st);
}

}  // namespace specdec
