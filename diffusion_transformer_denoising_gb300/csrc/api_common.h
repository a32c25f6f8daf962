// What the translation units of the C ABI share: the error state of the
// calling thread and the status-returning check macros.
#pragma once
#include <cuda_runtime.h>

#include "../../include/dit.h"

namespace dit {

// Records the message dit_last_error() returns on this thread and returns s.
dit_status fail(dit_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Forgets the calling thread's message (first line of an entry point).
void clear_last_error();

}  // namespace dit

#define CU_TRY(expr)                                                                                    \
  do {                                                                                                  \
    cudaError_t e_ = (expr);                                                                            \
    if (e_ != cudaSuccess) return fail(DIT_ERR_CUDA, "%s failed: %s", #expr, cudaGetErrorString(e_)); \
  } while (0)
#define DIT_TRY(expr)                 \
  do {                                \
    dit_status s_ = (expr);           \
    if (s_ != DIT_OK) return s_;      \
  } while (0)
