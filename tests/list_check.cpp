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
