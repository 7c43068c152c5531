// The work list that gpb_attend_plan_build writes and the attention kernels
// read, and the shapes both agree on.
#pragma once

#include <algorithm>

#include "row_format.h"

namespace gpb {

// One workgroup: query rows [row0, row0 + n_rows) of one KV head over n_tiles
// tiles of keys.  A query row is token * G + head within the KV head's group
// of G heads, so the heads that share keys are neighbours.  Tile v is tile0 +
// v for v < n_first and tile1 + v - n_first after it (a window leaves out the
// keys between the first tokens and itself); keys outside [key_lo, key_hi)
// are masked.  With partial >= 0 the item's sums go to that row of the
// workspace, else its results go out.
struct AttendItem {
  int32_t req, row0, n_rows, kv_head;
  int32_t key_lo, key_hi, n_tiles, tile0;
  int32_t n_first, tile1, partial, wide;
  int32_t pos_min, pos_max, pad0, pad1;
};

// Rows [row0, row0 + n_rows) of one KV head, all of one token, whose parts
// start at workspace rows refs[ref0 .. ref0 + n_refs).
struct AttendJoin {
  int32_t row0, n_rows, kv_head, ref0, n_refs, pad0, pad1, pad2;
};

constexpr int kItemInts = sizeof(AttendItem) / 4;
constexpr int kJoinInts = sizeof(AttendJoin) / 4;

// Query rows of an item of attention kernel `which` (0: 64-wide heads, 1: 128,
// 2: latent rows).  A wide item's four waves take a quarter of the rows each of
// one tile of 64 keys (over latent rows two waves share a half); a narrow
// item's four waves hold the same rows, each over tiles of 32 keys of its own.
// Rows that fit a narrow item are one: 8 queries over a window of 4096 keys, 64
// heads over 8, 64 wide, take 21.9 us so and 43 us as wide items; one query over
// 737 keys, 128 wide, 13.7 and 16.6.  Batches of narrow items alone have a
// kernel of their own, whose registers are theirs: 21.9 us, and 32.7 in the
// kernel that has both.
constexpr int kNarrowRows = 32;
constexpr int rows_of(int which, bool wide) {
  return which == 2 ? 64 : !wide ? kNarrowRows : which == 0 ? 256 : 128;
}
constexpr int kWideTile = 64, kNarrowTile = 32;

// Which attention kernel a format has, or -1.
inline int attend_kernel(const gpb_row_format &f) {
  if (f.k_dim == 64 && f.v_dim == 64 && !f.values_in_key) return 0;
  if (f.k_dim == 128 && f.v_dim == 128 && !f.values_in_key) return 1;
  if (f.k_dim == 576 && f.v_dim == 512 && f.values_in_key) return 2;
  return -1;
}

// Workgroups a CU holds of attention kernel `which`, by the registers that a
// wave's rows take.
constexpr int blocks_per_cu(int which) { return which == 2 ? 1 : 2; }

struct AttendArgs {
  const int32_t *list;
  const uint16_t *q;
  int64_t q_ts, q_hs;
  const uint8_t *rows;      // dense buffer or pool
  int64_t n_rows;           // rows of it; paged: of its whole pages
  const int32_t *pages;     // NULL: dense
  const int32_t *base;      // k_bases (dense), page_base or NULL (paged)
  int64_t n_listed, pages_stride;
  uint16_t *out;
  int64_t o_ts, o_hs;
  float *lse;
  float *sums, *ml;         // workspace: sums [partial rows][DV], (m, l) pairs
  int32_t *status;
  float c;                  // scale * log2(e)
  int32_t row_bytes, page_rows, page_shift, n_pages, window, sinks;
  int32_t G, hkv, n_heads, n_tokens, bs, max_keys;
  int32_t n_items, n_joins, n_refs, n_partial_rows, joins_at, refs_at, positions_at;
};

// What the kernels take from a plan as it is.
inline void plan_args(const gpb_attend_plan &p, AttendArgs *a) {
  a->row_bytes = p.format.row_bytes; a->page_rows = p.page_rows;
  a->page_shift = p.page_rows & (p.page_rows - 1) ? -1 : __builtin_ctz(p.page_rows);
  // (no position reaches 2^30, so a larger window is no window)
  a->window = std::min(p.window, 1 << 30); a->sinks = std::min(p.sinks, 1 << 30);
  a->hkv = p.format.n_kv_heads; a->n_heads = p.n_heads; a->G = p.n_heads / a->hkv;
  a->n_tokens = p.n_tokens; a->bs = p.bs; a->max_keys = p.max_keys;
  a->n_items = p.n_items; a->n_joins = p.n_joins; a->n_refs = p.n_refs;
  a->n_partial_rows = p.n_partial_rows;
  a->joins_at = p.joins_at; a->refs_at = p.refs_at; a->positions_at = p.positions_at;
}

// Whether an item lies in the batch.  The list is the caller's device memory:
// the kernel leaves out an item that does not, whatever it holds.
__host__ __device__ inline bool item_fits(const AttendArgs &a, const AttendItem &it, int which,
                                          bool narrow) {
  const int64_t all = static_cast<int64_t>(a.n_tokens) * a.G;
  return it.req >= 0 && it.req < a.bs && it.row0 >= 0 && it.n_rows >= 1 &&
         it.n_rows <= rows_of(which, it.wide) && !(narrow && it.wide) &&
         static_cast<int64_t>(it.row0) + it.n_rows <= all &&
         it.kv_head >= 0 && it.kv_head < a.hkv && it.key_lo >= 0 &&
         it.key_lo <= it.key_hi && it.key_hi <= a.max_keys &&
         (it.n_tiles == 0 || it.key_lo < it.key_hi) && it.n_tiles >= 0 &&
         it.n_tiles <= a.max_keys / kNarrowTile + 1 && it.n_first >= 0 &&
         it.tile0 >= 0 && it.tile1 >= 0 && it.tile0 <= a.max_keys / kNarrowTile &&
         it.tile1 <= a.max_keys / kNarrowTile && it.partial >= -1 &&
         it.partial <= a.n_partial_rows - (it.partial < 0 ? 0 : it.n_rows);
}

// Which keys of an item are read.
struct AttendKeys {
  int lo, last;
  int sunk, near, behind;  // keys [sunk, near) are read as `behind`

  __host__ __device__ AttendKeys(const AttendArgs &a, const AttendItem &it)
      : lo(it.key_lo), last(std::max(std::min(it.key_hi - 1, it.pos_max), lo)), sunk(0), near(0),
        behind(0) {
    if (a.window > 0) {
      sunk = a.sinks;
      near = std::max(lo, it.pos_min + 1 - a.window);
      // (shared keys may all lie behind the window but for the first tokens)
      if (near > last) last = std::max(std::min(last, sunk - 1), lo);
      behind = near;
    }
  }
  // The key, or if no row sees it one that some row sees (an item that has
  // tiles has such a one): the pages behind a window and past the last query
  // may no longer, or not yet, be the request's.
  __host__ __device__ int in_range(int key) const {
    key = std::max(key, lo);
    return std::min(key >= sunk && key < near ? behind : key, last);
  }
};

}  // namespace gpb
