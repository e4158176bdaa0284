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
//   4 rows  bf16 11.5 12.9 / 174 176 / 87 86 / 128 141, e4m3 12.5 15.2 / 184 199 / 83 82 / 153 196
//   12      bf16 13.1 12.9 / 174 179 / 90 88 / 144 143, e4m3 13.7 15.4 / 187 205 / 84 84 / 169 198
//   16      bf16 13.1 13.1 / 175 180 / 91 88 / 148 142, e4m3 14.1 15.4 / 189 206 / 84 85 / 174 198
//   20      bf16 13.5 13.1 / 334 181 / 158 88 / 259 144, e4m3 14.3 15.2 / 356 206 / 150 85 / 313 200
// The average decides: in a batch of one large request among many small ones, the
// large one takes a tile of 16 rows at a time.
constexpr int kWarpRows = 16;

// Which kernel serves a call.
enum class Kernel { kWarp, kTile, kWide };

constexpr int kTileRows = 128;   // rows of a tile of the tile kernel

// The wide kernel (cross_wide.cu) reads a key for 256 rows, and is bound by the products; the
// tile kernel divides a call's rows among more CTAs.  Tile and wide kernel, device us, 32
// query and 8 kv heads of 128, bf16 states (rows of a request and kv head; f16 the same within
// 4 %), and of 64:
//   1 request, 2816 states    128  22 22    160  21 23    256  21 26    512  24 27
//   8 of 2816                 128  37 38    160  42 41    384  58 60    512  72 63
//   64 of 1500                128 100 103   160 156 115   256 176 123   512 324 210
//   64: 8 of 2816             128  26 29    160  36 32    384  46 48    512  56 48
//       64 of 1500            128  74 90    160 121 95    256 126 99    512 228 169
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
