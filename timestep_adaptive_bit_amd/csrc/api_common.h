// Helpers of the extern "C" entry points: error records on a context, HIP
// status translation, pointer alignment.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "../../include/tabit.h"
#include "tabit_internal.h"

namespace {

int fail(tabit_ctx* ctx, int status, const char* fmt, ...) {
  if (ctx != nullptr) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    ctx->err = buf;
  }
  return status;
}

int hip_status(tabit_ctx* ctx, hipError_t e, const char* what) {
  if (e == hipSuccess) return TABIT_OK;
  return fail(ctx, TABIT_EHIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
