// host.hpp -- host-side helpers shared by the translation units of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/metis.h"

namespace metis {

// Sets the message of metis_last_error() and returns the status.
__attribute__((format(printf, 2, 3))) metis_status fail(metis_status st, const char* fmt, ...);

// Once per device, with that device current: its tables and status word.
metis_status ensure_device_tables();

// The current device's numeric status word (after ensure_device_tables).
int* device_status();

// Carves a caller's workspace; with a null base it only counts.
struct Carver {
  char* base;
  size_t off = 0;
  size_t cap;
  explicit Carver(void* b, size_t c) : base((char*)b), cap(c) {}
  template <typename T>
  T* take(size_t count) {
    off = (off + 255) & ~(size_t)255;
    T* p = base ? (T*)(base + off) : nullptr;
    off += count * sizeof(T);
    return p;
  }
  size_t used() const { return (off + 255) & ~(size_t)255; }
};

inline int64_t round_up64(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

inline bool dtype_ok(int32_t dt) { return dt == METIS_BF16 || dt == METIS_F32; }

#define HIP_TRY(expr)                                                                     \
  do {                                                                                    \
    hipError_t e__ = (expr);                                                              \
    if (e__ != hipSuccess) return fail(METIS_E_HIP, "%s: %s", #expr, hipGetErrorString(e__)); \
  } while (0)

#define LAUNCH_CHECK()                                                                    \
  do {                                                                                    \
    hipError_t e__ = hipGetLastError();                                                   \
    if (e__ != hipSuccess) return fail(METIS_E_HIP, "kernel launch: %s", hipGetErrorString(e__)); \
  } while (0)

}  // namespace metis
