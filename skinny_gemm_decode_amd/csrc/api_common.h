// What the ABI's source files share: error reporting and the device check
// (defined in api.hip).
#pragma once

#include <stdint.h>

#include "skg.h"

namespace skg {

// Records the calling thread's message and returns st / clears it.
skg_status fail(skg_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
skg_status ok();

// SKG_E_DEVICE unless the current device is gfx950; its CU count.
skg_status check_device(int* cus = nullptr);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace skg
