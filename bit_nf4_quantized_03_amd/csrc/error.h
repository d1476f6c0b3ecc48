// Status and message of a C entry point, shared by the files that define
// entry points (the message is what qlora_last_error returns).
#pragma once

#include <hip/hip_runtime.h>

namespace qnf4 {

// Records the formatted message for the calling thread and returns `status`.
int api_fail(int status, const char *fmt, ...);
// QLORA_OK, or QLORA_ERR_HIP with the HIP error's name behind `where`.
int api_hip_status(hipError_t e, const char *where);

}  // namespace qnf4
