// abi_common.h - what the C entry points share: the calling thread's last error, and checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

// Records the description gdn_last_error returns (printf-style) and hands back `s`.
gdn_status fail(gdn_status s, const char* fmt, ...);
gdn_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace gdn
