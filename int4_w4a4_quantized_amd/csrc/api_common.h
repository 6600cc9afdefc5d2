// What the sources of the C ABI share: the thread's error text and the device
// check, defined in ck4_api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/ck4.h"

namespace ck4 {

// Sets ck4_last_error() and returns s.
ck4_status api_fail(ck4_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// CK4_OK if the current device is a gfx950, else CK4_ERR_DEVICE. Its number
// goes to *dev if dev is not null.
ck4_status api_check_device(const char *fn, int *dev);
// The status of a launch: CK4_OK clears ck4_last_error().
ck4_status api_launched(const char *fn, hipError_t e);

}  // namespace ck4
