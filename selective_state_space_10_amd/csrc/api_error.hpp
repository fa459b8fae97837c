// api_error.hpp -- the calling thread's last error message, shared by the
// C-ABI files (it lives in ssm_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

namespace ssm {

void api_clear_error();
// Stores the message and returns the status.
__attribute__((format(printf, 2, 3))) int api_fail(int status, const char *fmt, ...);
int api_hip_status(hipError_t e, const char *what);

}  // namespace ssm
