// Host-side pieces shared by the argument checks of every entry point: the
// calling thread's error message, descriptor checks and HIP error codes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <string>

#include "kda_recoverssm.h"

namespace kda {
namespace host {

inline thread_local std::string g_err;

__attribute__((format(printf, 2, 3)))
inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return code;
}

inline int elem_size(int32_t dt) {
  return dt == KDA_F32 ? 4 : (dt == KDA_BF16 ? 2 : 0);
}

inline bool aligned(const void* p, uintptr_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

inline const char* dt_name(int32_t dt) {
  return dt == KDA_F32 ? "float32" : (dt == KDA_BF16 ? "bfloat16" : "?");
}

inline bool supported_head_dim(int64_t d) {
  return d == 16 || d == 32 || d == 64 || d == 128;
}

// Checks ndim, non-negative sizes, known dtype and a data pointer.
inline int check_desc(const kda_tensor& t, const char* name, int ndim) {
  if (t.ndim != ndim)
    return fail(KDA_E_SHAPE, "%s must have %d dimensions (got %d)", name,
                ndim, t.ndim);
  for (int i = 0; i < ndim; ++i)
    if (t.shape[i] < 0)
      return fail(KDA_E_SHAPE, "%s has a negative size", name);
  if (elem_size(t.dtype) == 0)
    return fail(KDA_E_DTYPE, "%s has an unknown dtype code %d", name,
                t.dtype);
  int64_t numel = 1;
  for (int i = 0; i < ndim; ++i) numel *= t.shape[i];
  if (t.data == nullptr && numel > 0)
    return fail(KDA_E_ARG, "%s has no data pointer", name);
  return KDA_OK;
}

inline bool shape_is(const kda_tensor& t, int64_t a, int64_t b, int64_t c = -1,
              int64_t d = -1) {
  if (t.shape[0] != a || t.shape[1] != b) return false;
  if (c >= 0 && t.shape[2] != c) return false;
  if (d >= 0 && t.shape[3] != d) return false;
  return true;
}

inline int device_status(int hip_rc, const char* what) {
  if (hip_rc == 0) return KDA_OK;
  return fail(KDA_E_DEVICE, "%s: HIP error %d (%s)", what, hip_rc,
              hipGetErrorString(hipError_t(hip_rc)));
}

}  // namespace host
}  // namespace kda

#define KDA_TRY(expr)             \
  do {                            \
    int rc_ = (expr);             \
    if (rc_ != KDA_OK) return rc_; \
  } while (0)
