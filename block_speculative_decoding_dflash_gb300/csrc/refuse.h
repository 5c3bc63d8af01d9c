// What the C entries share: refusals with a message, and pointer checks.
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "dflash.h"
#include "kernels.h"

namespace dfl {

void set_global_error(const char* msg);

inline int refuse(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    set_global_error(buf);
  } catch (...) {
  }
  return code;
}

inline int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return DFLASH_OK;
  return refuse(DFLASH_ECUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

// A device array that a call needs: not NULL and aligned to `bytes`. An array that is
// read or written an element at a time may be a slice of a larger one, which may
// start anywhere.
inline int need_aligned(const char* call, const void* p, const char* name, unsigned bytes) {
  if (!p) return refuse(DFLASH_EINVAL, "%s: %s is NULL", call, name);
  if (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) return refuse(DFLASH_EINVAL, "%s: %s is not %u-byte aligned", call, name, bytes);
  return DFLASH_OK;
}

}  // namespace dfl

#define PG(call)          \
  do {                    \
    int rc_ = (call);     \
    if (rc_) return rc_;  \
  } while (0)
