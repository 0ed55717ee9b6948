// What the C-ABI translation units share: the error report of a call, its
// checks and its workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lora_mi355x.h"
#include "trace.hpp"

namespace lora {

// Records the calling thread's error text (lora_last_error) and returns s.
lora_status fail(lora_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

#define CHECK(cond, status, ...)          \
  do {                                    \
    if (!(cond)) return ::lora::fail(status, __VA_ARGS__); \
  } while (0)

#define LAUNCH(expr)                                                              \
  do {                                                                            \
    hipError_t e_ = (expr);                                                       \
    if (e_ != hipSuccess) return ::lora::fail(LORA_EDEVICE, "%s: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

// LAUNCH with the launch bracketed for lora_trace_* under `name`.
#define LAUNCHN(name, stream, expr)       \
  do {                                    \
    ::lora::TraceScope ts_(name, stream); \
    LAUNCH(expr);                         \
  } while (0)

#define TRY(expr)                    \
  do {                               \
    lora_status s_ = (expr);         \
    if (s_ != LORA_OK) return s_;    \
  } while (0)

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

// Bump allocator over the caller's workspace (256-byte aligned pieces).
struct Ws {
  char* base;
  size_t off = 0;
  explicit Ws(void* b) : base(static_cast<char*>(b)) {}
  void* take(size_t bytes) {
    off = (off + 255) & ~(size_t)255;
    void* p = base ? base + off : nullptr;
    off += bytes;
    return p;
  }
};

inline lora_status check_ws(const void* ws, size_t have, size_t need) {
  CHECK(have >= need, LORA_EWORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", have, need);
  CHECK(need == 0 || ws != nullptr, LORA_EWORKSPACE, "workspace is NULL");
  CHECK(aligned(ws, 16), LORA_EALIGN, "workspace is not 16-byte aligned");
  return LORA_OK;
}

}  // namespace lora
