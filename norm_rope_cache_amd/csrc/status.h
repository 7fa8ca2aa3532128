// What the C entry points share (defined in api.cpp): the thread's error
// text, the current device's compute units, the status of a launch.
#pragma once

#include <stdint.h>

namespace nrc {

// Sets nrc_last_error's text and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// CUs of the current device.
int num_cus();

// NRC_OK for rc == 0, else NRC_EIO with the runtime's error as the text.
int launch_status(int rc, const char* what);

}  // namespace nrc
