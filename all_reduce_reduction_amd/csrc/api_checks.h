// api_checks.h -- argument checks shared by the entry points that work on rows
// and arrays of one rank (api_loss.cpp, api_layer.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "simar.h"

namespace simar {

constexpr int64_t kMaxBytes = (int64_t)1 << 46;
constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;

inline bool float_dtype(int d) { return d == SIM_FP32 || d == SIM_FP16 || d == SIM_BF16; }
inline int64_t size_of(int d) { return d == SIM_FP32 ? 4 : 2; }

// An array of a call: its address range (first to last element), the alignment
// its elements need, and for rows with others' elements between them the bytes
// of a row and from one to the next.
struct Array {
  const void* p;
  int64_t bytes;
  int64_t align;
  bool output;
  int64_t width = 0, pitch = 0;
};

inline Array rows_of(const void* p, int64_t rows, int64_t cols, int64_t stride, int dtype, bool output) {
  const int64_t e = size_of(dtype);
  return {p, rows > 0 ? ((rows - 1) * stride + cols) * e : 0, e, output, cols * e, stride * e};
}

inline bool rows_fit(int64_t rows, int64_t cols, int64_t stride) {
  return rows >= 0 && cols >= 1 && stride >= cols && stride <= kMaxBytes / 4 &&
         (rows == 0 || rows <= kMaxBytes / 4 / stride);
}

// Whether two arrays share a byte.  Rows at the same distances may lie between
// each other's: column slices of one wide buffer.
inline bool overlap(const Array& a, const Array& b) {
  const uintptr_t p = (uintptr_t)a.p, q = (uintptr_t)b.p;
  if (!(p < q + (uintptr_t)b.bytes && q < p + (uintptr_t)a.bytes)) return false;
  if (a.pitch == 0 || a.pitch != b.pitch) return true;
  const int64_t to_b = p <= q ? (int64_t)((q - p) % (uintptr_t)a.pitch)
                              : (a.pitch - (int64_t)((p - q) % (uintptr_t)a.pitch)) % a.pitch;
  return to_b < a.width || to_b + b.width > a.pitch;
}

// An output that may lie exactly on an input: same address, same rows.
struct Over {
  int output, input;
};

// NULL arrays are absent ones.
template <int N, int M>
int check_arrays(const Array (&a)[N], const Over (&may)[M]) {
  for (const Array& v : a)
    if ((uintptr_t)v.p & (uintptr_t)(v.align - 1)) return SIM_ERR_ALIGN;
  for (int i = 0; i < N; i++) {
    if (!a[i].p || !a[i].output || a[i].bytes == 0) continue;
    for (int j = 0; j < N; j++) {
      if (j == i || !a[j].p || a[j].bytes == 0) continue;
      bool allowed = false;
      for (const Over& o : may)
        allowed = allowed || (o.output == i && o.input == j && a[i].p == a[j].p && a[i].pitch == a[j].pitch &&
                              a[i].width == a[j].width);
      if (!allowed && overlap(a[i], a[j])) return SIM_ERR_ALIAS;
    }
  }
  return SIM_OK;
}
template <int N>
int check_arrays(const Array (&a)[N]) {
  const Over none[] = {{-1, -1}};
  return check_arrays(a, none);
}

// Too many rows for a launch are the caller's error.  It is always a call's
// first launch that has too many: the others are only made for few rows, or
// with as many threads as the first.
inline int hip_status(hipError_t e) {
  return e == hipSuccess ? SIM_OK : e == hipErrorInvalidConfiguration ? SIM_ERR_INVALID_ARG : SIM_ERR_HIP;
}

// A call's scratch.
inline int check_work(const void* work, size_t have, int64_t need, int64_t align = 4) {
  if (need == 0) return SIM_OK;
  if (!work) return SIM_ERR_INVALID_ARG;
  if ((uintptr_t)work & (uintptr_t)(align - 1)) return SIM_ERR_ALIGN;
  return have < (size_t)need ? SIM_ERR_NOMEM : SIM_OK;
}

}  // namespace simar
