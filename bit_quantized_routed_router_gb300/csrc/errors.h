// Errors at the C ABI: a status code and a message in the caller's buffer.
#pragma once
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/ds_moe.h"

namespace dsm {

inline int fail(char *err, size_t errlen, int code, const char *fmt, ...) {
  if (err && errlen) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(err, errlen, fmt, ap);
    va_end(ap);
  }
  return code;
}

inline int cuda_fail(char *err, size_t errlen, cudaError_t e, const char *what) {
  return fail(err, errlen, DS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace dsm
