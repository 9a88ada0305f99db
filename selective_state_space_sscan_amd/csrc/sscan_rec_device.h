// sscan_rec_device.h -- the arithmetic of the gated recurrence that its kernels share.
#pragma once

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "sscan_rec.h"

// Products and sums are joined only where the code says so: otherwise the kernels, which are
// built for many combinations of arguments, would round the same token differently.
#pragma clang fp contract(off)

namespace sscan {
namespace rec {

typedef __bf16 bf16;

constexpr float kLog2e = 1.44269504088896340736f;

// By the hardware's exp2 and reciprocal, a unit in the last place each: off by at most
// (1.25 |x| + 5) 2^-24 of the value.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e));
}

// A channel's constant c softplus(lam).  softplus(x) = max(x, 0) + log1p(w), w = exp(-|x|)
// by an exponent in two parts; log1p(w) is the logarithm of the rounded sum s = 1 + w plus
// the rounding's error w - (s - 1), off by less than a unit in the last place.
__device__ __forceinline__ float decay_rate(const float* lam, int64_t ch, float c) {
  // far out w is 0 and not the difference of infinities; a NaN stays one
  const float l = lam[ch], x = l < -200.0f || l > 200.0f ? -200.0f : -fabsf(l), t = x * kLog2e;
  const float low = fmaf(x, kLog2e, -t) + x * 1.925963033500e-8f;  // what the product and the constant drop
  const float e = __builtin_amdgcn_exp2f(t), w = fmaf(e * low, 0.693147181f, e), s = 1.0f + w;
  const float rate = c * (fmaxf(l, 0.0f) + fmaf(__builtin_amdgcn_logf(s), 0.693147181f, w - (s - 1.0f)));
  return rate > FLT_MAX ? FLT_MAX : rate;  // decays to 0 as well, and its product with a slope of 0 is 0
}

// 1 - exp(-m) for |m| < 1/4: by its series (the next term is below 2^-28 of the sum).
__device__ __forceinline__ float small_loss(float m) {
  float p = fmaf(m, -1.0f / 5040, 1.0f / 720);
  p = fmaf(m, -p, 1.0f / 120);
  p = fmaf(m, p, -1.0f / 24);
  p = fmaf(m, p, 1.0f / 6);
  p = fmaf(m, p, -0.5f);
  return m * fmaf(m, p, 1.0f);
}

// 1 - exp(-m): where the difference would lose digits by the series.  Decays near 1 are taken
// as 1 minus this: their rounding is what a long sum of states sees of them.  `far`: whether
// any channel of the wave decays that fast at all (its rate, the largest m of its tokens,
// reaches 1/4); where none does, the exponential is passed over.
__device__ __forceinline__ float decay_loss(float m, bool far) {
  float p = small_loss(m);
  if (far) p = fabsf(m) < 0.25f ? p : 1.0f - __builtin_amdgcn_exp2f(m * -kLog2e);
  return p;
}

// The decay of a token: a, and with lam also 1 - a and w = sqrt(1 - a^2).
struct Decay {
  float a, loss, w;
};

template <bool GATED>
__device__ __forceinline__ Decay decay(float g, float rate, bool far) {
  if constexpr (GATED) {
    const float loss = decay_loss(rate * sigmoid(g), far);
    return {1.0f - loss, loss, __builtin_amdgcn_sqrtf(loss * (2.0f - loss))};
  } else {
    // -inf: m = inf, whose series is not taken
    return {fabsf(g) < 0.25f ? 1.0f - small_loss(-g) : __builtin_amdgcn_exp2f(g * kLog2e), 0.0f, 1.0f};
  }
}

// Whether a wave has a channel whose rate reaches 1/4 (or is no number).
template <int C>
__device__ __forceinline__ bool any_far(const float (&rate)[C]) {
  bool far = false;
#pragma unroll
  for (int c = 0; c < C; ++c) far = far || !(rate[c] < 0.25f);
  return __ballot(far) != 0;
}

}  // namespace rec
}  // namespace sscan
