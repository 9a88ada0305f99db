// sscan_norm.hip -- RMS norms of a block fused with what stands beside them: a
// mixer's heads normed with their silu gate, and the residual scale and sum with the
// next block's norm.  All of them are bound by HBM: a group of TPR threads holds one
// normed vector in registers (eight elements a thread), so every input is read once
// and every output written once; blocks walk over rows, so that the weights are loaded
// once per block and the next row's values while a row is reduced.  Sums and norms are
// float32.  The gradients of the weights are summed per thread over a block's rows, across
// the block in LDS and over the blocks by a second kernel, always in the same order.
// Measured, where a large copy moves 5.1 TB/s: norm and gate of 16384 x 16 x 128 bf16 5.8 TB/s
// (part stays in the cache), its gradients at 8192 x 1536 4.1 (3.5 with the sums over blocks),
// residual norm gradients of 16384 x 1536 5.2 (4.8).
#include "sscan_delta.h"

#include "sscan_delta_device.h"

namespace sscan {
namespace norm {

using delta::bf16;
using delta::bf16x8;
using delta::f32x4;
using delta::f32x8;

// Blocks that walk over the rows.  Forward, 16384 x 16 x 128 bf16: 8192 blocks 34.9 us, 4096
// 36.5.  Backward each block leaves a row of partial sums: gated norm, 8192 x 1536 bf16,
// 1024 blocks 30.9 us, 512 38.7; residual norm with a post norm (three rows of sums and
// 157 registers a thread: 512 blocks are most of what fits) 512 blocks 87 us, 1024 100.
constexpr int kMaxBlocks = 8192, kMaxGatedBackBlocks = 1024, kMaxAddBackBlocks = 512;

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

// By the hardware's exp2 and reciprocal, a unit in the last place (2^-23) each: the gradients'
// kernel would otherwise spend as long on expf and the division as on its memory traffic.
// The error is at most (1.25 |z| + 5) 2^-24 of the value: 1.25 |z| from the exponent z log2 e
// (the constant and the product rounded, times ln 2), 2 each from exp2 and the reciprocal, 1
// from the sum.  Float32 calls have it too.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}

// A group's walk over the units (row, head) first, first + step, ...: divided once, then
// advanced by the step's quotient and remainder.
struct UnitWalk {
  int64_t u, row, h, units, heads, step, step_rows, step_heads;

  __device__ __forceinline__ UnitWalk(int64_t first, int64_t step_, int64_t units_, int64_t heads_)
      : u(first), units(units_), heads(heads_), step(step_) {
    row = heads == 1 ? u : u / heads;
    h = heads == 1 ? 0 : u % heads;
    step_rows = heads == 1 ? step : step / heads;
    step_heads = heads == 1 ? 0 : step % heads;
  }
  __device__ __forceinline__ bool live() const { return u < units; }
  __device__ __forceinline__ void next() {
    u += step;
    row += step_rows;
    h += step_heads;
    if (h >= heads) {
      h -= heads;
      ++row;
    }
  }
};

// ---- norm and gate of a mixer's heads -------------------------------------------------
//   y = x r w silu(z), r = 1 / rms(x)           (gate after the norm)
//   y = m r w, m = x silu(z), r = 1 / rms(m)    (gate_first)
template <typename IO, int TPR, bool whole>
__global__ __launch_bounds__(threads<TPR>()) void gated_norm_kernel(GatedNormArgs a) {
  __shared__ float lds[2][3][16];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  const int64_t units = a.rows * a.heads, step = int64_t(gridDim.x) * kGroups;
  UnitWalk at(int64_t(blockIdx.x) * kGroups + grp, step, units, a.heads);
  float w[8], next_x[8], next_z[8], next_w[8];
  const auto load_next = [&] {
    const int size = at.live() ? int(a.size) : 0;
    load<whole>(static_cast<const IO*>(a.x) + at.row * a.xr + at.h * a.xh, size, t, next_x);
    load<whole>(static_cast<const IO*>(a.z) + at.row * a.zr + at.h * a.zh, size, t, next_z);
    if (a.per_head) load<whole>(a.weight + at.h * a.size, size, t, next_w);
  };
  if (!a.per_head) load_or<whole>(a.weight, int(a.size), t, 1.0f, w);
  load_next();
  const float inv = 1.0f / float(a.size);
  int turn = 0;
  for (int64_t u0 = int64_t(blockIdx.x) * kGroups; u0 < units; u0 += step) {
    float x[8], z[8], ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = next_x[j];
      z[j] = next_z[j];
      if (a.per_head) w[j] = next_w[j];
    }
    const int size = at.live() ? int(a.size) : 0;
    IO* out = static_cast<IO*>(a.out) + at.u * a.size;
    at.next();
    load_next();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[j] *= sigmoid(z[j]);
      if (a.gate_first) x[j] *= z[j];
      ss[0] += x[j] * x[j];
    }
    group_sum<TPR>(ss, lds, turn);
    turn ^= 1;
    const float r = 1.0f / sqrtf(ss[0] * inv + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= a.gate_first ? r * w[j] : r * w[j] * z[j];
    store<whole>(out, size, t, x);
  }
}

// With n = m r the gradient at m is r (dn - m r^2 mean(dn m)).  Per block: all units
// (shared weight), or the units of head blockIdx % heads (per_head).
template <typename IO, int TPR, bool whole>
__global__ __launch_bounds__(threads<TPR>()) void gated_norm_bwd_kernel(GatedNormArgs a, float* partial) {
  __shared__ float lds[2][3][16];
  __shared__ float sums[partial_lds<TPR>()];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  const int64_t sets = a.per_head ? a.heads : 1;  // heads told apart
  const int64_t set = int64_t(blockIdx.x) % sets, first = int64_t(blockIdx.x) / sets * kGroups;
  const int64_t units = a.per_head ? a.rows : a.rows * a.heads, step = int64_t(gridDim.x) / sets * kGroups;
  UnitWalk at(first + grp, step, units, a.per_head ? 1 : a.heads);
  float w[8], dw[8] = {}, next_x[8], next_z[8], next_d[8];
  const auto load_next = [&] {
    const int size = at.live() ? int(a.size) : 0;
    const int64_t h = a.per_head ? set : at.h;
    load<whole>(static_cast<const IO*>(a.x) + at.row * a.xr + h * a.xh, size, t, next_x);
    load<whole>(static_cast<const IO*>(a.z) + at.row * a.zr + h * a.zh, size, t, next_z);
    load<whole>(static_cast<const IO*>(a.dout) + (at.row * a.heads + h) * a.size, size, t, next_d);
  };
  load_or<whole>(a.weight ? a.weight + set * a.size : nullptr, int(a.size), t, 1.0f, w);
  load_next();
  const float inv = 1.0f / float(a.size);
  int turn = 0;
  for (int64_t u0 = first; u0 < units; u0 += step) {
    float x[8], z[8], d[8], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = next_x[j];
      z[j] = next_z[j];
      d[j] = next_d[j];
    }
    const int size = at.live() ? int(a.size) : 0;
    const int64_t flat = (at.row * a.heads + (a.per_head ? set : at.h)) * a.size;
    at.next();
    load_next();
    float sig[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sig[j] = sigmoid(z[j]);
      const float gate = z[j] * sig[j];
      const float m = a.gate_first ? x[j] * gate : x[j];
      const float dn = a.gate_first ? d[j] * w[j] : d[j] * w[j] * gate;
      sum[0] += m * m;
      sum[1] += dn * m;
    }
    group_sum<TPR>(sum, lds, turn);
    turn ^= 1;
    const float r = 1.0f / sqrtf(sum[0] * inv + a.eps), mean = sum[1] * inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gate = z[j] * sig[j], slope = sig[j] * (1.0f + z[j] * (1.0f - sig[j]));
      if (a.gate_first) {
        const float m = x[j] * gate, dm = r * (d[j] * w[j] - m * (r * r) * mean);
        dw[j] += d[j] * m * r;
        z[j] = dm * x[j] * slope;
        x[j] = dm * gate;
      } else {
        const float n = x[j] * r;
        dw[j] += d[j] * gate * n;
        z[j] = d[j] * n * w[j] * slope;
        x[j] = r * (d[j] * w[j] * gate - x[j] * (r * r) * mean);
      }
    }
    store<whole>(static_cast<IO*>(a.dx) + flat, size, t, x);
    store<whole>(static_cast<IO*>(a.dz) + flat, size, t, z);
  }
  if (a.dweight) write_partial<TPR, whole>(partial + int64_t(blockIdx.x) * a.size, int(a.size), t, dw, sums);
}

// ---- residual scale and sum with the next norm ----------------------------------------
//   total = residual + scale a, a = x or x / rms(x) * post_weight; out = total / rms(total) * weight
// The norm is taken of the total as it is stored, so that the backward pass (which
// reads the stored total) differentiates what was computed.
template <typename IO, typename RES, int TPR, bool whole>
__global__ __launch_bounds__(threads<TPR>()) void add_norm_kernel(AddNormArgs a) {
  __shared__ float lds[2][3][16];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  const int64_t step = int64_t(gridDim.x) * kGroups;
  float w[8], sc[8], pw[8], next_x[8], next_y[8];
  const auto load_next = [&](int64_t u) {
    const int size = u < a.rows ? int(a.size) : 0;
    const int64_t flat = size ? u * a.size : 0;
    load<whole>(static_cast<const IO*>(a.x) + flat, size, t, next_x);
    load<whole>(static_cast<const RES*>(a.residual) + flat, a.residual ? size : 0, t, next_y);
  };
  load_next(int64_t(blockIdx.x) * kGroups + grp);
  load_or<whole>(a.weight, int(a.size), t, 1.0f, w);
  load_or<whole>(a.scale, int(a.size), t, 1.0f, sc);
  load_or<whole>(a.post_weight, int(a.size), t, 1.0f, pw);
  const float inv = 1.0f / float(a.size);
  int turn = 0;
  for (int64_t u0 = int64_t(blockIdx.x) * kGroups; u0 < a.rows; u0 += step) {
    const int64_t u = u0 + grp, flat = u * a.size;
    const int size = u < a.rows ? int(a.size) : 0;
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = next_x[j];
      y[j] = next_y[j];
    }
    load_next(u + step);
    if (a.post_weight) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += x[j] * x[j];
      group_sum<TPR>(ss, lds, turn);
      turn ^= 1;
      const float r = 1.0f / sqrtf(ss[0] * inv + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= r * pw[j];
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = float(RES(y[j] + x[j] * sc[j]));
      ss[0] += y[j] * y[j];
    }
    store<whole>(static_cast<RES*>(a.residual_out) + flat, size, t, y);
    group_sum<TPR>(ss, lds, turn);
    turn ^= 1;
    const float r = 1.0f / sqrtf(ss[0] * inv + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= r * w[j];
    store<whole>(static_cast<IO*>(a.out) + flat, size, t, y);
  }
}

// POST: with a norm of x itself.  Sums left by a block: dweight, dscale, dpost_weight.
// Blocks of 1024 threads have 128 registers a thread: they read the vectors per row.
template <typename IO, typename RES, int TPR, bool whole, bool POST>
__global__ __launch_bounds__(threads<TPR>()) void add_norm_bwd_kernel(AddNormArgs a, float* partial) {
  __shared__ float lds[2][3][16];
  __shared__ float sums[partial_lds<TPR>()];
  constexpr int kGroups = threads<TPR>() / TPR;
  constexpr bool kHold = TPR < 1024;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  const int64_t step = int64_t(gridDim.x) * kGroups;
  float w[8], sc[8], pw[8], dw[8] = {}, ds[8] = {}, dp[8] = {};
  float next_x[8], next_y[8], next_d[8], next_e[8];
  const auto load_next = [&](int64_t u) {
    const int size = u < a.rows ? int(a.size) : 0;
    const int64_t flat = size ? u * a.size : 0;
    load<whole>(static_cast<const IO*>(a.x) + flat, size, t, next_x);
    load<whole>(static_cast<const RES*>(a.residual) + flat, size, t, next_y);
    load<whole>(static_cast<const IO*>(a.dout) + flat, size, t, next_d);
    load<whole>(static_cast<const RES*>(a.dresidual_out) + flat, a.dresidual_out ? size : 0, t, next_e);
  };
  const auto load_vectors = [&] {
    load_or<whole>(a.weight, int(a.size), t, 1.0f, w);
    load_or<whole>(a.scale, int(a.size), t, 1.0f, sc);
    if (POST) load_or<whole>(a.post_weight, int(a.size), t, 1.0f, pw);
  };
  if (kHold) {
    load_next(int64_t(blockIdx.x) * kGroups + grp);
    load_vectors();
  }
  const float inv = 1.0f / float(a.size);
  int turn = 0;
  for (int64_t u0 = int64_t(blockIdx.x) * kGroups; u0 < a.rows; u0 += step) {
    const int64_t u = u0 + grp, flat = u * a.size;
    const int size = u < a.rows ? int(a.size) : 0;
    if (!kHold) {
      load_next(u);
      load_vectors();
    }
    float x[8], y[8], d[8], e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = next_x[j];
      y[j] = next_y[j];
      d[j] = next_d[j];
      e[j] = next_e[j];
    }
    if (kHold) load_next(u + step);
    float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum[0] += y[j] * y[j];
      sum[1] += d[j] * w[j] * y[j];
      if (POST) sum[2] += x[j] * x[j];
    }
    group_sum<TPR>(sum, lds, turn);
    turn ^= 1;
    const float r = 1.0f / sqrtf(sum[0] * inv + a.eps), mean = sum[1] * inv;
    const float rx = POST ? 1.0f / sqrtf(sum[2] * inv + a.eps) : 1.0f;
    float dot[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] += d[j] * y[j] * r;
      e[j] += r * (d[j] * w[j] - y[j] * (r * r) * mean);  // gradient of the total
      const float n = x[j] * rx, scaled = e[j] * sc[j];
      if (POST) {
        ds[j] += e[j] * n * pw[j];
        dp[j] += scaled * n;
        d[j] = scaled * pw[j];
        dot[0] += d[j] * x[j];
      } else {
        ds[j] += e[j] * x[j];
        d[j] = scaled;
      }
    }
    store<whole>(static_cast<RES*>(a.dresidual) + flat, size, t, e);
    if (POST) {
      group_sum<TPR>(dot, lds, turn);
      turn ^= 1;
      const float m2 = dot[0] * inv;
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rx * (d[j] - x[j] * (rx * rx) * m2);
    }
    store<whole>(static_cast<IO*>(a.dx) + flat, size, t, d);
  }
  float* dst = partial + int64_t(blockIdx.x) * 3 * a.size;
  if (a.dweight) write_partial<TPR, whole>(dst, int(a.size), t, dw, sums);
  if (a.dscale) write_partial<TPR, whole>(dst + a.size, int(a.size), t, ds, sums);
  if (POST && a.dpost_weight) write_partial<TPR, whole>(dst + 2 * a.size, int(a.size), t, dp, sums);
}

// out[set][e] = sum over the blocks of set `set` of partial[block][part][e], in order:
// blocks set, set + sets, ... of nblocks; 64 slices of the blocks per element.
struct SumArgs {
  const float* partial;
  float* out[3];
  int64_t size, pitch, nblocks, sets, first;  // first: sets before this launch's
};

// Most blocks of a launch in x: per-head weights of 65536 heads of 1024 need 2^22, whose 2^32
// threads no launch takes.
constexpr int kSumCols = 16, kSumSlices = 64, kMaxSumBlocks = 1 << 20;

__global__ __launch_bounds__(1024) void partial_sum_kernel(SumArgs s) {
  __shared__ float lds[kSumSlices][kSumCols];
  const int lane = int(threadIdx.x) % kSumCols, slice = int(threadIdx.x) / kSumCols;
  const int64_t nb = (s.size + kSumCols - 1) / kSumCols;
  const int64_t set = s.first + int64_t(blockIdx.x) / nb, e = int64_t(blockIdx.x) % nb * kSumCols + lane;
  const int part = int(blockIdx.y);
  if (!s.out[part]) return;
  const int64_t per_set = s.nblocks / s.sets;
  float x = 0.0f;
  if (e < s.size)
#pragma unroll 8
    for (int64_t k = slice; k < per_set; k += kSumSlices)
      x += s.partial[(set + k * s.sets) * s.pitch + part * s.size + e];
  lds[slice][lane] = x;
  __syncthreads();
#pragma unroll
  for (int half = kSumSlices / 2; half > 0; half /= 2) {
    if (slice < half) lds[slice][lane] += lds[slice + half][lane];
    __syncthreads();
  }
  if (slice == 0 && e < s.size) s.out[part][set * s.size + e] = lds[0][lane];
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads that hold one vector of this size: the smallest power of two (16 or more)
// whose eight elements each suffice.
int threads_of(int64_t size) {
  int t = 16;
  while (int64_t(t) * 8 < size) t *= 2;
  return t;
}

int64_t back_blocks(int64_t units, int64_t size, int64_t heads, int64_t limit) {
  const int64_t groups = threads_of(size) < 256 ? 256 / threads_of(size) : 1;
  if (heads == 0) return 0;
  const int64_t most = limit > heads ? limit / heads : 1;
  const int64_t want = div_up(units, groups);
  return (want < most ? want : most) * heads;
}

hipError_t launch_sums(SumArgs s, int parts, hipStream_t stream) {
  const int64_t nb = div_up(s.size, kSumCols), most = kMaxSumBlocks / nb;  // nb <= 512
  for (s.first = 0; s.first < s.sets; s.first += most) {
    const int64_t sets = s.sets - s.first < most ? s.sets - s.first : most;
    partial_sum_kernel<<<dim3(unsigned(sets * nb), unsigned(parts)), 1024, 0, stream>>>(s);
  }
  return hipGetLastError();
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

using norm::bf16;

size_t gated_norm_bwd_workspace(int64_t rows, int64_t heads, int64_t size) {
  // whichever of the shared and the per-head weight needs more blocks
  const int64_t a = norm::back_blocks(rows * heads, size, 1, norm::kMaxGatedBackBlocks),
                b = heads > kNormMaxHeads ? 0 : norm::back_blocks(rows, size, heads, norm::kMaxGatedBackBlocks);
  return size_t(a > b ? a : b) * size_t(size) * 4;
}

size_t add_norm_bwd_workspace(int64_t rows, int64_t size) {
  return size_t(norm::back_blocks(rows, size, 1, norm::kMaxAddBackBlocks)) * 3 * size_t(size) * 4;
}

template <typename IO>
static hipError_t gated_fwd(const GatedNormArgs& a, hipStream_t stream) {
  return norm::by_shape(a.size, [&](auto tpr, auto whole) {
    constexpr int T = decltype(tpr)::value, B = norm::threads<T>();
    int64_t n = norm::div_up(a.rows * a.heads, B / T);
    if (n > norm::kMaxBlocks) n = norm::kMaxBlocks;
    norm::gated_norm_kernel<IO, T, decltype(whole)::value><<<dim3(unsigned(n)), B, 0, stream>>>(a);
  });
}

template <typename IO>
static hipError_t gated_bwd(const GatedNormArgs& a, float* ws, hipStream_t stream) {
  const int64_t sets = a.per_head ? a.heads : 1;
  const int64_t n = norm::back_blocks(a.per_head ? a.rows : a.rows * a.heads, a.size, sets, norm::kMaxGatedBackBlocks);
  if (sets == 0) return hipSuccess;  // per-head weights of no heads
  // without rows there are no blocks, and the sums over none are zeros
  const hipError_t e = n == 0 ? hipSuccess : norm::by_shape(a.size, [&](auto tpr, auto whole) {
    constexpr int T = decltype(tpr)::value, B = norm::threads<T>();
    norm::gated_norm_bwd_kernel<IO, T, decltype(whole)::value><<<dim3(unsigned(n)), B, 0, stream>>>(a, ws);
  });
  if (e != hipSuccess || !a.dweight) return e;
  return norm::launch_sums({ws, {a.dweight, nullptr, nullptr}, a.size, a.size, n, sets, 0}, 1, stream);
}

template <typename IO, typename RES>
static hipError_t add_fwd(const AddNormArgs& a, hipStream_t stream) {
  return norm::by_shape(a.size, [&](auto tpr, auto whole) {
    constexpr int T = decltype(tpr)::value, B = norm::threads<T>();
    int64_t n = norm::div_up(a.rows, B / T);
    if (n > norm::kMaxBlocks) n = norm::kMaxBlocks;
    norm::add_norm_kernel<IO, RES, T, decltype(whole)::value><<<dim3(unsigned(n)), B, 0, stream>>>(a);
  });
}

template <typename IO, typename RES>
static hipError_t add_bwd(const AddNormArgs& a, float* ws, hipStream_t stream) {
  const int64_t n = norm::back_blocks(a.rows, a.size, 1, norm::kMaxAddBackBlocks);
  const hipError_t e = n == 0 ? hipSuccess : norm::by_shape(a.size, [&](auto tpr, auto whole) {
    constexpr int T = decltype(tpr)::value, B = norm::threads<T>();
    const dim3 grid{unsigned(n)};
    if (a.post_weight)
      norm::add_norm_bwd_kernel<IO, RES, T, decltype(whole)::value, true><<<grid, B, 0, stream>>>(a, ws);
    else
      norm::add_norm_bwd_kernel<IO, RES, T, decltype(whole)::value, false><<<grid, B, 0, stream>>>(a, ws);
  });
  if (e != hipSuccess || !(a.dweight || a.dscale || a.dpost_weight)) return e;
  return norm::launch_sums({ws, {a.dweight, a.dscale, a.dpost_weight}, a.size, 3 * a.size, n, 1, 0}, 3, stream);
}

// Heads that continue each other in memory are rows, where their weight is shared.
static GatedNormArgs collapsed(GatedNormArgs a) {
  if (!a.per_head && a.heads > 1 && a.xr == a.heads * a.xh && a.zr == a.heads * a.zh) {
    a.rows *= a.heads;
    a.heads = 1;
    a.xr = a.xh;
    a.zr = a.zh;
  }
  return a;
}

hipError_t launch_gated_norm(const GatedNormArgs& args, hipStream_t stream) {
  const GatedNormArgs a = collapsed(args);
  return a.io_bf16 ? gated_fwd<bf16>(a, stream) : gated_fwd<float>(a, stream);
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs& args, float* ws, hipStream_t stream) {
  const GatedNormArgs a = collapsed(args);
  return a.io_bf16 ? gated_bwd<bf16>(a, ws, stream) : gated_bwd<float>(a, ws, stream);
}

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream) {
  if (a.io_bf16) return a.res_bf16 ? add_fwd<bf16, bf16>(a, stream) : add_fwd<bf16, float>(a, stream);
  return a.res_bf16 ? add_fwd<float, bf16>(a, stream) : add_fwd<float, float>(a, stream);
}

hipError_t launch_add_norm_bwd(const AddNormArgs& a, float* ws, hipStream_t stream) {
  if (a.io_bf16) return a.res_bf16 ? add_bwd<bf16, bf16>(a, ws, stream) : add_bwd<bf16, float>(a, ws, stream);
  return a.res_bf16 ? add_bwd<float, bf16>(a, ws, stream) : add_bwd<float, float>(a, ws, stream);
}

}  // namespace sscan
