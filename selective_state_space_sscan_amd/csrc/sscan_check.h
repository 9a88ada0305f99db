// sscan_check.h -- what the argument checks of the C ABI share: alignment, the ranges of
// memory that tensors cover, products of sizes that do not overflow.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "sscan.h"

namespace sscan {
namespace check {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return p ? Range{lo, lo + bytes} : Range{0, 0};
}

inline bool overlap(const Range& a, const Range& b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline bool clash(const Range& out, std::initializer_list<Range> others) {
  for (const Range& r : others)
    if (overlap(out, r)) return true;
  return false;
}

constexpr int64_t kMaxElems = int64_t(1) << 50;

// a * b * ..., or -1 beyond 2^50.
inline int64_t product(std::initializer_list<int64_t> f) {
  int64_t n = 1;
  for (int64_t x : f)
    if (__builtin_mul_overflow(n, x, &n) || n > kMaxElems) return -1;
  return n;
}

// Elements from the first to one past the last of a strided view whose last `size`
// elements are contiguous, or -1 (a negative stride, or beyond 2^50).
inline int64_t extent(const int64_t* dims, const int64_t* strides, int n, int64_t size) {
  int64_t last = size;
  for (int i = 0; i < n; ++i) {
    if (strides[i] < 0) return -1;
    if (dims[i] <= 1) continue;
    int64_t step = 0;
    if (__builtin_mul_overflow(dims[i] - 1, strides[i], &step) || __builtin_add_overflow(last, step, &last) ||
        last > kMaxElems)
      return -1;
  }
  return last;
}

inline bool dtype_ok(int d) { return d == SSCAN_F32 || d == SSCAN_BF16; }
inline size_t dtype_size(int d) { return d == SSCAN_BF16 ? 2 : 4; }

inline int check_workspace(const void* workspace, size_t have, size_t need, size_t align) {
  if (need == 0) return SSCAN_OK;
  if (!workspace || have < need) return SSCAN_ERR_WORKSPACE;
  return aligned(workspace, align) ? SSCAN_OK : SSCAN_ERR_ALIGN;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? SSCAN_OK : SSCAN_ERR_HIP; }

}  // namespace check
}  // namespace sscan
