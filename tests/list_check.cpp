// Every item of a work list as the attention kernels take it, on the CPU: the
// test by which they leave items out, and the keys they read.
#include <cstdint>

#include "attend.h"

using namespace gpb;

// 0, or 1 where an item would be left out; *item is its number.
extern "C" int list_items_fit(const gpb_attend_plan *plan, const int32_t *list, int32_t *item) {
  AttendArgs a = {};
  plan_args(*plan, &a);
  const int which = attend_kernel(plan->format);
  const AttendItem *it = reinterpret_cast<const AttendItem *>(list);
  for (int32_t i = 0; i < plan->n_items; ++i)
    if (!item_fits(a, it[i], which, which != 2 && plan->n_wide == 0)) {
      *item = i;
      return 1;
    }
  return 0;
}

// 0, or 1 where an item with tiles reads a key that none of its rows sees.
// The key read in place of one past the last tile is the item's first.
extern "C" int list_keys_seen(const gpb_attend_plan *plan, const int32_t *list, int32_t *item) {
  AttendArgs a = {};
  plan_args(*plan, &a);
  const AttendItem *items = reinterpret_cast<const AttendItem *>(list);
  for (int32_t i = 0; i < plan->n_items; ++i) {
    const AttendItem &it = items[i];
    const AttendKeys keys(a, it);
    const int tile = it.wide ? kWideTile : kNarrowTile;
    const auto seen = [&](int key) {
      if (key < it.key_lo || key >= it.key_hi) return false;
      for (int row = 0; row < it.n_rows; row += row + a.G < it.n_rows ? a.G : 1) {
        const int pos = list[a.positions_at + (it.row0 + row) / a.G];
        if (key <= pos && (a.window == 0 || pos - key < a.window || key < a.sinks)) return true;
      }
      return false;
    };
    int last = -1;  // (the same key again says nothing new)
    for (int v = 0; v < it.n_tiles; ++v) {
      const int first = (v < it.n_first ? it.tile0 + v : it.tile1 + v - it.n_first) * tile;
      for (int x = -1; x < tile; ++x) {
        const int key = keys.in_range(x < 0 ? keys.lo : first + x);
        if (key != last && !seen(key)) {
          *item = i;
          return 1;
        }
        last = key;
      }
    }
  }
  return 0;
}
