// attend_held.hip -- the attention kernels of rows held in 8 bits (gfx950).
#include "attend_kernel.h"

namespace gpb {

int launch_attend_held(int type, int which, const AttendArgs &a, bool narrow,
                       hipStream_t stream) {
  return type == GPB_BF16 ? launch_format<__bf16, true>(which, a, narrow, stream)
                          : launch_format<_Float16, true>(which, a, narrow, stream);
}

}  // namespace gpb
