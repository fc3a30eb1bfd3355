// Host helpers the C ABI's source files share.  Not installed; not part of
// the ABI.
#pragma once

#include <hip/hip_runtime_api.h>

#include "fpstok.h"

#define FPSTOK_API extern "C" __attribute__((visibility("default")))

namespace fpstok {

// Records the detail of a failed call for fpstok_last_error and returns `st`.
fpstok_status fail(fpstok_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the detail and returns FPSTOK_OK.
fpstok_status ok();
fpstok_status hip_fail(hipError_t e, const char* what);

}  // namespace fpstok
