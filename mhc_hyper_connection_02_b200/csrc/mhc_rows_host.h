// Host-side checks shared by the row operators' entry points (layer norm, token log probabilities,
// distillation). Part of the library's single translation unit, after mhc_api.cu.
#pragma once

#include <type_traits>

#include "mhc.h"
#include "mhc_internal.h"

namespace mhc {

// Makes the device that owns `p` current for a call and puts the caller's device back at its end.
struct DeviceScope {
  int status;
  int before = -1;
  explicit DeviceScope(const void* p) {
    if (cudaGetDevice(&before) != cudaSuccess) before = -1;
    status = bind_device(p);
  }
  ~DeviceScope() {
    int now = -1;
    if (before >= 0 && cudaGetDevice(&now) == cudaSuccess && now != before) cudaSetDevice(before);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;
};

// A refused launch is reported once, as this call's status: it leaves no error behind for the next.
inline int launched(int status) {
  if (status != MHC_OK) cudaGetLastError();
  return status;
}

inline bool dtype_ok(int dtype) {
  return dtype == MHC_DTYPE_BF16 || dtype == MHC_DTYPE_F16 || dtype == MHC_DTYPE_F32;
}
inline size_t dtype_size(int dtype) { return dtype == MHC_DTYPE_F32 ? 4 : 2; }
inline bool misaligned(const void* p, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0;
}

// T rows of n elements, `stride` elements apart: positions inside a row fit an int with room for
// a block's step, and byte offsets fit 63 bits.
inline bool rows_ok(int64_t T, int64_t n, int64_t stride) {
  return n > 0 && n <= (int64_t(1) << 28) && stride >= n && stride <= (int64_t(1) << 40) &&
         T <= (int64_t(1) << 31) - 1 && mul_ok(T, stride, INT64_MAX / 16);
}
// Bytes from the first element of the first row to the end of the last row.
inline size_t row_bytes(int64_t T, int64_t n, int64_t stride, size_t size) {
  return T > 0 ? static_cast<size_t>((T - 1) * stride + n) * size : 0;
}

struct Range {
  const void* p;  // null: no such array
  size_t n;
};
inline bool overlap(const Range& a, const Range& b) {
  return a.p && b.p && overlaps(a.p, a.n, b.p, b.n);
}
// Does any output overlap an input or another output?
inline bool any_overlap(const Range* outs, int n_out, const Range* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

}  // namespace mhc
