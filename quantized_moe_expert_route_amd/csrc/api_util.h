// Argument checks shared by the C entry points (host code).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "qmoe.h"

namespace qmoe {

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Device that owns a device pointer, or -1.
inline int ptr_device(const void* p) {
  hipPointerAttribute_t a;
  if (hipPointerGetAttributes(&a, p) != hipSuccess) {
    (void)hipGetLastError();
    return -1;
  }
  if (a.type != hipMemoryTypeDevice && a.type != hipMemoryTypeManaged) return -1;
  return a.device;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) { ok = false; return; }
    if (prev != dev && hipSetDevice(dev) != hipSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

constexpr int64_t kMaxRows = (int64_t)1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 40;  // elements between rows: kMaxRows of them stay below 2^63 bytes

inline bool type16(int t) { return t == MOE_BF16 || t == MOE_FP16; }
inline size_t type_bytes(int t) { return t == MOE_FP32 ? 4 : 2; }

// Bytes from a [rows, cols] tensor's first element to behind its last.
inline size_t span(int64_t rows, int64_t ld, int64_t cols, size_t elem) {
  return rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * elem : 0;
}

// The device of gfx950 pointers `ptrs`, all on one: MOE_OK and *dev, *cus.
inline moe_status device_of(const void* const* ptrs, int n, int* dev, int* cus) {
  const int d = ptr_device(ptrs[0]);
  if (d < 0) return MOE_ERR_DEVICE;
  for (int i = 1; i < n; ++i)
    if (ptrs[i] && ptr_device(ptrs[i]) != d) return MOE_ERR_DEVICE;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, d) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ERR_DEVICE;
  }
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0) return MOE_ERR_DEVICE;
  *dev = d;
  *cus = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 256;
  return MOE_OK;
}

// The current device, which must be a gfx950.
inline moe_status current_device(int* dev, int* cus) {
  hipDeviceProp_t prop;
  int d;
  if (hipGetDevice(&d) != hipSuccess || hipGetDeviceProperties(&prop, d) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ERR_DEVICE;
  }
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0) return MOE_ERR_DEVICE;
  *dev = d;
  *cus = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 256;
  return MOE_OK;
}

// A workspace of at least `need` bytes.
inline moe_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  return ws && ((uintptr_t)ws & 255) == 0 && have >= need ? MOE_OK : MOE_ERR_WORKSPACE;
}

// A buffer of a call: outputs must overlap no other buffer of it.
struct Buf {
  const void* p;
  size_t bytes;
  bool out;
};
inline moe_status check_buffers(const Buf* b, int n, int device) {
  for (int i = 0; i < n; ++i)
    if (b[i].p && b[i].bytes)
      for (int j = 0; j < n; ++j)
        if (j != i && b[i].out && b[j].p && b[j].bytes && overlaps(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
          return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (b[i].p && b[i].bytes && ptr_device(b[i].p) != device) return MOE_ERR_DEVICE;
  return MOE_OK;
}

}  // namespace qmoe
