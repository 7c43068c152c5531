// The work list that gpb_attend_plan_build writes and the attention kernels
// read, and the shapes both agree on.
#pragma once

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

}  // namespace gpb
