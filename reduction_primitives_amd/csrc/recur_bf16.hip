// recur_bf16.hip -- the gated linear recurrence for one type of inputs (bf16).
#define RK_UNIT unit_recur_bf16
#include "rk_recur_kernels.hpp"

namespace rk {
int launch_recur_bf16(const RecurLaunch &L) { return launch_recur_x<bf16_in>(L); }
}  // namespace rk
