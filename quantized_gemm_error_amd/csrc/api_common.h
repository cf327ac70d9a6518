// Host helpers of the C ABI's entry points: status with a message, alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "internal.h"

namespace spear {

// Keeps `text` as this thread's last error and returns st.
spear_status_t set_last_error(spear_status_t st, const char *text);

namespace {

spear_status_t fail(spear_status_t st, const char *fmt, ...) {
  char text[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  return set_last_error(st, text);
}

spear_status_t ok() { return set_last_error(SPEAR_OK, ""); }

spear_status_t hip_status(hipError_t e, const char *what) {
  if (e != hipSuccess) return fail(SPEAR_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

#define TRY(expr)                                     \
  do {                                                \
    if (const spear_status_t st_ = (expr)) return st_; \
  } while (0)

}  // namespace
}  // namespace spear
