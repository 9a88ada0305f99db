// sscan_pack8.h -- a block's scale and its elements in steps of it, for the kernels that keep
// activations in 8 bits.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sscan_rec.h"

#pragma clang fp contract(off)

namespace sscan {
namespace rec {

typedef __bf16 bf16;

// |x| as a whole number, in the order of the values: infinities above all numbers, NaN above them.
__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// From the largest magnitude of a block: its scale, and what turns elements into steps.  By
// float32 divisions, so that whoever repeats them has the same steps.
struct Scale {
  float step, per;
  __device__ __forceinline__ explicit Scale(unsigned m) {
    const float top = __uint_as_float(m);
    const bool fine = m < 0x7f800000u && top >= 0x1p-100f;
    per = fine ? 127.0f / top : 0.0f;
    step = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : fine ? top / 127.0f : 0.0f;
  }
  // 0 where the block has no scale
  __device__ __forceinline__ int steps(float x) const { return int(rintf(per == 0.0f ? 0.0f : x * per)); }
};

// The same with a scale's `per` alone.  A whole number of steps below 2^22 added to 1.5 2^23
// stands in the low bits of the sum, which is rounded as rintf is; bfloat16 has no NaN whose
// low bits are not 0.
template <typename IO>
__device__ __forceinline__ int8_t steps_of(float x, float per) {
  if constexpr (sizeof(IO) == 2) {
    const float y = x * per;
    return int8_t(__float_as_uint(y + 12582912.0f) & 0xffu);
  } else {
    return int8_t(int(rintf(per == 0.0f ? 0.0f : x * per)));
  }
}

}  // namespace rec
}  // namespace sscan
