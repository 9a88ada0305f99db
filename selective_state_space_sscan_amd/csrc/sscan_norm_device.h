// sscan_norm_device.h -- how the norms' kernels hold, load, store and sum rows: a group of
// TPR threads holds one vector in registers, eight elements a thread.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sscan_delta.h"
#include "sscan_delta_device.h"

namespace sscan {
namespace norm {

using delta::bf16;
using delta::bf16x8;
using delta::f32x4;
using delta::f32x8;

template <int TPR>
constexpr int threads() {
  return TPR < 256 ? 256 : TPR;
}

// Thread t holds elements 8 t .. 8 t + 7 of a vector, moved by 16-byte accesses at
// whatever alignment the rows have, which global memory takes (one element at a time,
// residual norm gradients of 8000 x 2001 took 166 us).  Where a size is no multiple of
// eight (not `whole`) the thread at its end reads the last eight elements instead, and
// takes for zeros the `dup` of them that its neighbour holds: loads of single elements
// would have to be waited for where they are put together, before the row ahead is
// reduced (99 us, so 78; 8000 x 2000 55).  In place, its neighbour may have stored them
// already: whatever it reads there is dropped.  Only its stores, and vectors of less than
// eight, go one element at a time.
struct Place {
  int off, dup;
};

template <bool whole>
__device__ __forceinline__ Place place(int size, int t) {
  if (whole || 8 * t + 8 <= size || size < 8) return {8 * t, 0};
  return {size - 8, 8 * t + 8 - size};
}

typedef bf16x8 bf16x8_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

__device__ __forceinline__ bf16x8 load_eight(const bf16* p) {
  return *reinterpret_cast<const bf16x8_any*>(p);
}

__device__ __forceinline__ f32x8 load_eight(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ void store_eight(bf16* p, bf16x8 x) { *reinterpret_cast<bf16x8_any*>(p) = x; }

__device__ __forceinline__ void store_eight(float* p, f32x8 x) {
  *reinterpret_cast<f32x4_any*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4_any*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}

// The vector's elements that thread t holds, zeros beyond its size.  Converted after the
// branches: inside them each would end with a wait for its load, and a row's loads would
// not be under way while the row before is reduced (residual norm gradients 119 us, so 92).
template <bool whole, typename T>
__device__ __forceinline__ void load(const T* p, int size, int t, float (&x)[8]) {
  const Place at = place<whole>(size, t);
  typename delta::Io<T>::V8 y = {};
  if (whole || size >= 8) {
    if (8 * t < size) y = load_eight(p + at.off);
  } else if (t == 0) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < size) y[j] = p[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = j < at.dup ? 0.0f : float(y[j]);
}

template <bool whole, typename T>
__device__ __forceinline__ void store(T* p, int size, int t, const float (&x)[8]) {
  const Place at = place<whole>(size, t);
  const int left = size - 8 * t;
  typename delta::Io<T>::V8 y;
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = T(x[j]);
  if (whole ? left > 0 : left >= 8) {
    store_eight(p + 8 * t, y);
  } else if (!whole && left > 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= at.dup && at.off + j < size) p[at.off + j] = y[j];
  }
}

template <bool whole>
__device__ __forceinline__ void load_or(const float* p, int size, int t, float missing, float (&x)[8]) {
  if (p) {
    load<whole>(p, size, t, x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = missing;
  }
}

// Sums over the TPR threads of a group, n of them at once; every thread of the block
// takes part.  Consecutive calls of a block alternate `turn`, so that one barrier a call
// is enough: a buffer is written again only after the barrier of the call between.
template <int TPR, int n>
__device__ __forceinline__ void group_sum(float (&x)[n], float (*lds)[3][16], int turn) {
#pragma unroll
  for (int k = 0; k < n; ++k)
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m *= 2) x[k] += __shfl_xor(x[k], m);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    const int wave = int(threadIdx.x) >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < n; ++k) lds[turn][k][wave] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < n; ++k) {
      x[k] = lds[turn][k][wave / kWaves * kWaves];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) x[k] += lds[turn][k][wave / kWaves * kWaves + w];
    }
  }
}

// Adds the groups' sums of one block in order and writes them as the block's partial.
template <int TPR, bool whole>
__device__ __forceinline__ void write_partial(float* dst, int size, int t, const float (&x)[8], float* lds) {
  if constexpr (TPR >= 256) {
    store<whole>(dst, size, t, x);
  } else {
    constexpr int kGroups = 256 / TPR, kCap = TPR * 8;
    const int grp = int(threadIdx.x) / TPR;
    const Place at = place<whole>(size, t);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= at.dup) lds[grp * kCap + at.off + j] = x[j];
    __syncthreads();
    for (int e = int(threadIdx.x); e < kCap; e += 256) {
      float s = 0.0f;
      for (int g = 0; g < kGroups; ++g) s += lds[g * kCap + e];
      if (e < size) dst[e] = s;
    }
  }
}

template <int TPR>
constexpr int partial_lds() {
  return TPR >= 256 ? 16 : 256 * 8;
}

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads that hold one vector of this size: the smallest power of two (16 or more)
// whose eight elements each suffice.
inline int threads_of(int64_t size) {
  int t = 16;
  while (int64_t(t) * 8 < size) t *= 2;
  return t;
}

template <int TPR, typename F>
void by_end(int64_t size, F f) {
  if (size % 8 == 0)
    f(std::integral_constant<int, TPR>(), std::true_type());
  else
    f(std::integral_constant<int, TPR>(), std::false_type());
}

// f(threads a vector, whole), as constants.
template <typename F>
hipError_t by_shape(int64_t size, F f) {
  switch (threads_of(size)) {
    case 16: by_end<16>(size, f); break;
    case 32: by_end<32>(size, f); break;
    case 64: by_end<64>(size, f); break;
    case 128: by_end<128>(size, f); break;
    case 256: by_end<256>(size, f); break;
    case 512: by_end<512>(size, f); break;
    default: by_end<1024>(size, f); break;  // size <= kNormMaxSize
  }
  return hipGetLastError();
}

}  // namespace norm
}  // namespace sscan
