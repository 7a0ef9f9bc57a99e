// og_host.hpp -- what the C-ABI translation units share on the host: the
// calling thread's stream and error text, and the device check
// (og_api.hip defines them).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "og.h"

namespace og::host {

// Records the message and returns `code`.
og_status fail(og_status code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message and returns OG_OK.
og_status ok();
// OG_OK when the current device is a gfx950.
og_status check_device();
// OG_OK, or the error of the launches since the last check.
og_status check_launch(const char *what);
// The calling thread's stream.
hipStream_t current_stream();

}  // namespace og::host
