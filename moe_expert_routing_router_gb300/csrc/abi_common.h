// Host-side state that the files of the C ABI share (defined in abi.cu).
#pragma once

#include <stdint.h>

#include "moe_router.h"

namespace moe {

// Records the calling thread's error message and returns `s`.
moe_status abi_fail(moe_status s, const char* message);
// SM count of the current device.
moe_status abi_sms(int* sms);
// Limit of the bounded device waits, and the arrivals that the tests of an
// expired wait add to a barrier (moe_set_unreachable_barriers).
uint64_t abi_wait_ns();
unsigned abi_barrier_extra();

}  // namespace moe
