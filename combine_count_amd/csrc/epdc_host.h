// Host helpers shared by the files that define entry points (epdc_api.cpp,
// epdc_api_ops.cpp).  Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "../../include/epdc.h"

namespace epdc {
namespace host {

extern thread_local std::string g_lastError;  // what epdc_last_error returns

// Sets the thread's last error and returns `code`.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// EPDC_OK, or EPDC_ERR_HIP with the runtime's own message.
int hip_status(hipError_t e, const char *what);
// Validity of an epdc_cfg for numTokens tokens on the dispatch or combine leg.
int check_cfg(const epdc_cfg *c, int32_t numTokens, bool combine);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace host
}  // namespace epdc
