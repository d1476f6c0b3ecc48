// Status and message of a C entry point, shared by the files that define
// entry points (the message is what qlora_last_error returns).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/qlora_mx.h"

namespace qnf4 {

// Records the formatted message for the calling thread and returns `status`.
int api_fail(int status, const char *fmt, ...);
// QLORA_OK, or QLORA_ERR_HIP with the HIP error's name behind `where`.
int api_hip_status(hipError_t e, const char *where);
// The checks of a struct and its buffers; `name` is the argument in the message.
int api_check_weight(const qlora_nf4_weight *w, const char *fn);
int api_check_matrix(const char *fn, const char *name, const qlora_mx_matrix *q);

}  // namespace qnf4
