// entry.h -- argument checking shared by the C ABI entry points that have
// their own translation unit (adapters.cu, balance.cu, adamw.cu).
#pragma once

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include "moe_internal.h"

namespace moe {

// Records the message where moe_last_error() reads it and returns `code`.
inline int32_t entry_fail(int32_t code, const char* fmt, ...)
    __attribute__((format(printf, 2, 3)));
inline int32_t entry_fail(int32_t code, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  set_last_error(msg);
  return code;
}

inline bool ptr_aligned(const void* p, size_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// A launch's status as the entry point's.
inline int32_t entry_launched(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  return entry_fail(MOE_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(e));
}

constexpr size_t kWsAlign = 256;
constexpr size_t ws_up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }

}  // namespace moe
