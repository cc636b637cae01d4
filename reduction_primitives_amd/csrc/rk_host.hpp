// rk_host.hpp -- what rk_api.cpp shares with the other host files of the C
// ABI: the current device's size, the per-stream slots, the timing and
// failure hooks.
#pragma once

#include <cstdint>

namespace rk {
namespace host {

int device_cus();                     // compute units of the current device, 0 without one
int stream_slot(void *stream);        // the stream's slot of arrival counters, or -1
bool fused_finish();                  // rk_debug_set_fused_finish
bool injected_launch_failure();       // rk_debug_fail_launches
bool debug_enabled();                 // RK_DEBUG
void launch_events(void **begin, void **end);   // rk_debug_set_launch_events of this thread

}  // namespace host
}  // namespace rk
