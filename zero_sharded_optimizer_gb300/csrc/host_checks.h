// What the host sides of the vocabulary losses and of the embedding share: checks
// of pointers and buffers, and the workspace's layout.
#pragma once

#include <cstddef>
#include <cstdint>

#include "zero_gb300.h"

namespace zl {

// Sets the calling thread's error message and returns `code` (zero_host.cpp).
int set_error(int code, const char* fmt, ...);

inline int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

inline int elem_size(int32_t precision) { return precision == ZERO_FP32 ? 4 : 2; }

// A buffer the call touches: `rows` rows of `bytes` bytes, `stride` bytes apart.
struct Span {
  const void* p;
  int64_t rows, bytes, stride;
  const char* what;
  bool written;
};

// Whether two buffers share a byte. Rows of equal stride are compared by their
// phase, so that column blocks of one wider buffer pass.
inline bool overlap(const Span& x, const Span& y) {
  if (!x.p || !y.p || !x.rows || !y.rows || !x.bytes || !y.bytes) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  const uintptr_t a1 = a + uintptr_t((x.rows - 1) * x.stride + x.bytes);
  const uintptr_t b1 = b + uintptr_t((y.rows - 1) * y.stride + y.bytes);
  if (a1 <= b || b1 <= a) return false;
  if (x.stride == y.stride && x.rows > 1 && y.rows > 1) {
    const uintptr_t s = uintptr_t(x.stride);
    const uintptr_t d = b >= a ? (b - a) % s : (s - (a - b) % s) % s;
    if (d >= uintptr_t(x.bytes) && s - d >= uintptr_t(y.bytes)) return false;
  }
  return true;
}

inline int check_pointer(const void* ptr, int64_t count, size_t align, const char* what) {
  if (!ptr && count > 0) return set_error(ZERO_EINVAL, "%s is NULL", what);
  if (reinterpret_cast<uintptr_t>(ptr) % align)
    return set_error(ZERO_EALIGN, "%s is not aligned to %zu bytes", what, align);
  return ZERO_OK;
}

// Places the call's arrays in the workspace (base NULL: only counts bytes).
// Returns false when the size overflows.
struct Layout {
  uint8_t* base;
  int64_t at = 0;
  bool fits = true;
  template <typename T>
  T* take(int64_t count, int64_t times = 1) {
    const int64_t size = int64_t(sizeof(T));
    if (!fits || (times && count > (INT64_MAX / 4) / times / size)) {
      fits = false;
      return nullptr;
    }
    T* p = reinterpret_cast<T*>(base + at);
    at = round_up(at + count * times * size, 256);
    if (at > INT64_MAX / 4) fits = false;
    return p;
  }
};

}  // namespace zl
