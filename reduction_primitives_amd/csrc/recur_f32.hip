// recur_f32.hip -- the gated linear recurrence for one type of inputs (f32).
#define RK_UNIT unit_recur_f32
#include "rk_recur_kernels.hpp"

namespace rk {
int launch_recur_f32(const RecurLaunch &L) { return launch_recur_x<float>(L); }
}  // namespace rk
