// recur_f16.hip -- the gated linear recurrence for one type of inputs (f16).
#define RK_UNIT unit_recur_f16
#include "rk_recur_kernels.hpp"

namespace rk {
int launch_recur_f16(const RecurLaunch &L) { return launch_recur_x<f16_in>(L); }
}  // namespace rk
