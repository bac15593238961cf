// Host-side services of the C-ABI layer that its source files share: device
// check, call tag of the launch log, launch status and dispatch counters.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/convrot.h"

namespace cr {

// index of a counter in cr_counters.launches
enum HostEntry { HE_RQ = 0, HE_PACK = 1, HE_W4A4 = 2, HE_W4A8 = 3, HE_INT8 = 4, HE_LORA = 5, HE_ACT = 6 };

cr_status host_device_check();
// names the call for the launch log: its sizes and format arguments
void host_tag(const char* name, int64_t d0, int64_t d1, int64_t d2, int f0, int f1, int f2);
// the status of a call that enqueued `kernels` kernels with result `e`
cr_status host_finish(hipError_t e, HostEntry entry, uint64_t kernels);

inline bool host_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace cr
