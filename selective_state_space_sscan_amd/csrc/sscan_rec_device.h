// sscan_rec_device.h -- the arithmetic of the gated recurrence that its kernels share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sscan_rec.h"

namespace sscan {
namespace rec {

typedef __bf16 bf16;

constexpr float kLog2e = 1.44269504088896340736f;

// By the hardware's exp2 and reciprocal, a unit in the last place each: off by at most
// (1.25 |x| + 5) 2^-24 of the value.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e));
}

// A channel's constants: k = c softplus(lam) (with lam), by the library's exp and log1p.
__device__ __forceinline__ float decay_rate(const float* lam, int64_t ch, float c) {
  const float x = lam[ch];
  return c * (fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))));
}

// 1 - exp(-m): by its series up to m = 1/4 (the next term is below 2^-29 of the sum), where
// the difference would lose digits.  Decays near 1 are taken as 1 minus this: their
// rounding is what a long sum of states sees of them.
__device__ __forceinline__ float decay_loss(float m) {
  float p = fmaf(m, -1.0f / 7, 1.0f);
  p = fmaf(m * (-1.0f / 6), p, 1.0f);
  p = fmaf(m * (-1.0f / 5), p, 1.0f);
  p = fmaf(m * (-1.0f / 4), p, 1.0f);
  p = fmaf(m * (-1.0f / 3), p, 1.0f);
  p = fmaf(m * (-1.0f / 2), p, 1.0f);
  return fabsf(m) < 0.25f ? m * p : 1.0f - __builtin_amdgcn_exp2f(m * -kLog2e);
}

// The decay of a token: a, and with lam also 1 - a and w = sqrt(1 - a^2).
struct Decay {
  float a, loss, w;
};

template <bool GATED>
__device__ __forceinline__ Decay decay(float g, float rate) {
  if constexpr (GATED) {
    const float r = sigmoid(g), loss = decay_loss(rate * r);
    return {1.0f - loss, loss, __builtin_amdgcn_sqrtf(loss * (2.0f - loss))};
  } else {
    // -inf: m = inf, whose series is not taken
    return {fabsf(g) < 0.25f ? 1.0f - decay_loss(-g) : __builtin_amdgcn_exp2f(g * kLog2e), 0.0f, 1.0f};
  }
}

}  // namespace rec
}  // namespace sscan
