// mlp_error.h -- the calling thread's last error (mlp_last_error), shared by the C entry points.
#pragma once

#include <hip/hip_runtime_api.h>

namespace mlpk {

// Set the message (printf form) and return `code`.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear the message and return MLP_OK.
int ok();
// MLP_ERR_HIP with the runtime's text.
int hip_fail(hipError_t e, const char *what);

}  // namespace mlpk
