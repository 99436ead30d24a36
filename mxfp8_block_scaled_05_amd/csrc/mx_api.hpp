// Shared by the files of the C ABI (api.cpp, api_tokens.cpp): device check,
// launch status, enum bytes.  Defined in api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <string.h>

#include "mxfp8.h"

namespace mx {

// MXFP8_OK if the current device is gfx950; else the status to return.
mxfp8_status check_device();

// Status of a launch; keeps a failure's HIP code for mxfp8_last_hip_error.
mxfp8_status finish(hipError_t e);

// The integer a caller passed for an enum parameter.  C callers may pass any
// int; reading such a value through the enum type is undefined in C++ (the
// host UBSan build flags it), so enum arguments are validated on their bytes.
template <class E>
int raw(const E &e) {
    static_assert(sizeof(E) == sizeof(int), "enum arguments are int-sized");
    int v = 0;
    memcpy(&v, &e, sizeof v);
    return v;
}

}  // namespace mx
