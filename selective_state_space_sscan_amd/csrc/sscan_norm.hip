// sscan_norm.hip -- RMS norms of a block fused with what stands beside them: a
// mixer's heads normed with their silu gate, and the residual scale and sum with the
// next block's norm.  All of them are bound by HBM: a group of TPR threads holds one
// normed vector in registers (eight elements a thread), so every input is read once
// and every output written once, and blocks walk over rows so that the weights are
// loaded once per block.  Sums and norms are float32.  The gradients of
// the weights are summed per thread over a block's rows, across the block in LDS and
// over the blocks by a second kernel, always in the same order.
#include "sscan_delta.h"

#include "sscan_delta_device.h"

namespace sscan {
namespace norm {

using delta::bf16;
using delta::bf16x8;
using delta::f32x4;
using delta::f32x8;

constexpr int kMaxBlocks = 2048;     // forward: blocks that walk over the rows
constexpr int kMaxBackBlocks = 512;  // backward: each leaves one row of partial sums

template <int TPR>
constexpr int threads() {
  return TPR < 256 ? 256 : TPR;
}

// Element j of thread t: eight neighbours where 16-byte accesses are possible,
// otherwise neighbours across threads.
template <int TPR>
__device__ __forceinline__ int elem(int j, int t, bool wide) {
  return wide ? 8 * t + j : j * TPR + t;
}

template <typename T, int TPR>
__device__ __forceinline__ void load(const T* p, int size, int t, bool wide, float (&x)[8]) {
  if (wide) {
    const auto y = delta::load8(p + 8 * t, 8 * t < size ? 8 : 0, true);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = float(y[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j * TPR + t < size ? float(p[j * TPR + t]) : 0.0f;
  }
}

template <typename T, int TPR>
__device__ __forceinline__ void store(T* p, int size, int t, bool wide, const float (&x)[8]) {
  if (wide) {
    typename delta::Io<T>::V8 y;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = T(x[j]);
    if (8 * t < size) *reinterpret_cast<typename delta::Io<T>::V8*>(p + 8 * t) = y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * TPR + t < size) p[j * TPR + t] = T(x[j]);
  }
}

template <int TPR>
__device__ __forceinline__ void load_or(const float* p, int size, int t, bool wide, float missing, float (&x)[8]) {
  if (p) {
    load<float, TPR>(p, size, t, wide, x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = missing;
  }
}

// Sum over the TPR threads of a group; every thread of the block takes part.
template <int TPR>
__device__ __forceinline__ float group_sum(float x, float* lds) {
#pragma unroll
  for (int m = 1; m < (TPR < 64 ? TPR : 64); m *= 2) x += __shfl_xor(x, m);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    const int wave = int(threadIdx.x) >> 6;
    __syncthreads();  // the last sum's readers are done
    if ((threadIdx.x & 63) == 0) lds[wave] = x;
    __syncthreads();
    x = lds[wave / kWaves * kWaves];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) x += lds[wave / kWaves * kWaves + w];
  }
  return x;
}

// Adds the groups' sums of one block in order and writes them as the block's partial.
template <int TPR>
__device__ __forceinline__ void write_partial(float* dst, int size, int t, bool wide, const float (&x)[8], float* lds) {
  if constexpr (TPR >= 256) {
    store<float, TPR>(dst, size, t, wide, x);
  } else {
    constexpr int kGroups = 256 / TPR, kCap = TPR * 8;
    const int grp = int(threadIdx.x) / TPR;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[grp * kCap + elem<TPR>(j, t, wide)] = x[j];
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

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// ---- norm and gate of a mixer's heads -------------------------------------------------
//   y = x r w silu(z), r = 1 / rms(x)           (gate after the norm)
//   y = m r w, m = x silu(z), r = 1 / rms(m)    (gate_first)
template <typename IO, int TPR>
__global__ __launch_bounds__(threads<TPR>()) void gated_norm_kernel(GatedNormArgs a, bool wide) {
  __shared__ float lds[16];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  const int64_t units = a.rows * a.heads, step = int64_t(gridDim.x) * kGroups;
  float w[8];
  if (!a.per_head) load_or<TPR>(a.weight, a.size, t, wide, 1.0f, w);
  for (int64_t u0 = int64_t(blockIdx.x) * kGroups; u0 < units; u0 += step) {
    const int64_t u = u0 + grp;
    const bool live = u < units;
    const int64_t row = live ? u / a.heads : 0, h = live ? u % a.heads : 0;
    const int size = live ? int(a.size) : 0;
    float x[8], z[8];
    load<IO, TPR>(static_cast<const IO*>(a.x) + row * a.xr + h * a.xh, size, t, wide, x);
    load<IO, TPR>(static_cast<const IO*>(a.z) + row * a.zr + h * a.zh, size, t, wide, z);
    if (a.per_head) load<float, TPR>(a.weight + h * a.size, size, t, wide, w);
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[j] *= sigmoid(z[j]);
      if (a.gate_first) x[j] *= z[j];
      ss += x[j] * x[j];
    }
    const float r = 1.0f / sqrtf(group_sum<TPR>(ss, lds) / float(a.size) + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= a.gate_first ? r * w[j] : r * w[j] * z[j];
    store<IO, TPR>(static_cast<IO*>(a.out) + u * a.size, size, t, wide, x);
  }
}

// With n = m r the gradient at m is r (dn - m r^2 mean(dn m)).  Per block: all units
// (shared weight), or the units of head blockIdx % heads (per_head).
template <typename IO, int TPR>
__global__ __launch_bounds__(threads<TPR>()) void gated_norm_bwd_kernel(GatedNormArgs a, float* partial, bool wide) {
  __shared__ float lds[partial_lds<TPR>()];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  const int64_t heads = a.per_head ? a.heads : 1;  // heads told apart
  const int64_t head = int64_t(blockIdx.x) % heads;
  const int64_t units = a.per_head ? a.rows : a.rows * a.heads;
  const int64_t step = int64_t(gridDim.x) / heads * kGroups;
  float w[8], dw[8] = {};
  load_or<TPR>(a.weight ? a.weight + head * a.size : nullptr, a.size, t, wide, 1.0f, w);
  for (int64_t u0 = int64_t(blockIdx.x) / heads * kGroups; u0 < units; u0 += step) {
    const int64_t u = u0 + grp;
    const bool live = u < units;
    const int64_t row = !live ? 0 : a.per_head ? u : u / a.heads, h = !live ? 0 : a.per_head ? head : u % a.heads;
    const int size = live ? int(a.size) : 0;
    const int64_t flat = (row * a.heads + h) * a.size;
    float x[8], z[8], d[8];
    load<IO, TPR>(static_cast<const IO*>(a.x) + row * a.xr + h * a.xh, size, t, wide, x);
    load<IO, TPR>(static_cast<const IO*>(a.z) + row * a.zr + h * a.zh, size, t, wide, z);
    load<IO, TPR>(static_cast<const IO*>(a.dout) + flat, size, t, wide, d);
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sig = sigmoid(z[j]), gate = z[j] * sig;
      const float m = a.gate_first ? x[j] * gate : x[j];
      const float dn = a.gate_first ? d[j] * w[j] : d[j] * w[j] * gate;
      ss += m * m;
      dot += dn * m;
    }
    const float r = 1.0f / sqrtf(group_sum<TPR>(ss, lds) / float(a.size) + a.eps);
    const float mean = group_sum<TPR>(dot, lds) / float(a.size);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sig = sigmoid(z[j]), gate = z[j] * sig, slope = sig * (1.0f + z[j] * (1.0f - sig));
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
    store<IO, TPR>(static_cast<IO*>(a.dx) + flat, size, t, wide, x);
    store<IO, TPR>(static_cast<IO*>(a.dz) + flat, size, t, wide, z);
  }
  if (a.dweight) write_partial<TPR>(partial + int64_t(blockIdx.x) * a.size, a.size, t, wide, dw, lds);
}

// ---- residual scale and sum with the next norm ----------------------------------------
//   total = residual + scale a, a = x or x / rms(x) * post_weight; out = total / rms(total) * weight
// The norm is taken of the total as it is stored, so that the backward pass (which
// reads the stored total) differentiates what was computed.
template <typename IO, typename RES, int TPR>
__global__ __launch_bounds__(threads<TPR>()) void add_norm_kernel(AddNormArgs a, bool wide) {
  __shared__ float lds[16];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  float w[8], sc[8], pw[8];
  load_or<TPR>(a.weight, a.size, t, wide, 1.0f, w);
  load_or<TPR>(a.scale, a.size, t, wide, 1.0f, sc);
  load_or<TPR>(a.post_weight, a.size, t, wide, 1.0f, pw);
  for (int64_t u0 = int64_t(blockIdx.x) * kGroups; u0 < a.rows; u0 += int64_t(gridDim.x) * kGroups) {
    const bool live = u0 + grp < a.rows;
    const int64_t flat = (live ? u0 + grp : 0) * a.size;
    const int size = live ? int(a.size) : 0;
    float x[8], y[8];
    load<IO, TPR>(static_cast<const IO*>(a.x) + flat, size, t, wide, x);
    load<RES, TPR>(static_cast<const RES*>(a.residual) + flat, a.residual ? size : 0, t, wide, y);
    if (a.post_weight) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
      const float r = 1.0f / sqrtf(group_sum<TPR>(ss, lds) / float(a.size) + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= r * pw[j];
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = float(RES(y[j] + x[j] * sc[j]));
      ss += y[j] * y[j];
    }
    store<RES, TPR>(static_cast<RES*>(a.residual_out) + flat, size, t, wide, y);
    const float r = 1.0f / sqrtf(group_sum<TPR>(ss, lds) / float(a.size) + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= r * w[j];
    store<IO, TPR>(static_cast<IO*>(a.out) + flat, size, t, wide, y);
  }
}

// POST: with a norm of x itself.  Sums left by a block: dweight, dscale, dpost_weight.
template <typename IO, typename RES, int TPR, bool POST>
__global__ __launch_bounds__(threads<TPR>()) void add_norm_bwd_kernel(AddNormArgs a, float* partial, bool wide) {
  __shared__ float lds[partial_lds<TPR>()];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  float w[8], sc[8], pw[8], dw[8] = {}, ds[8] = {}, dp[8] = {};
  load_or<TPR>(a.weight, a.size, t, wide, 1.0f, w);
  load_or<TPR>(a.scale, a.size, t, wide, 1.0f, sc);
  if (POST) load_or<TPR>(a.post_weight, a.size, t, wide, 1.0f, pw);
  const float inv = 1.0f / float(a.size);
  for (int64_t u0 = int64_t(blockIdx.x) * kGroups; u0 < a.rows; u0 += int64_t(gridDim.x) * kGroups) {
    const bool live = u0 + grp < a.rows;
    const int64_t flat = (live ? u0 + grp : 0) * a.size;
    const int size = live ? int(a.size) : 0;
    float x[8], y[8], d[8], e[8];
    load<IO, TPR>(static_cast<const IO*>(a.x) + flat, size, t, wide, x);
    load<RES, TPR>(static_cast<const RES*>(a.residual) + flat, size, t, wide, y);
    load<IO, TPR>(static_cast<const IO*>(a.dout) + flat, size, t, wide, d);
    load<RES, TPR>(static_cast<const RES*>(a.dresidual_out) + flat, a.dresidual_out ? size : 0, t, wide, e);
    float ss = 0.0f, dot = 0.0f, xx = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ss += y[j] * y[j];
      dot += d[j] * w[j] * y[j];
      if (POST) xx += x[j] * x[j];
    }
    const float r = 1.0f / sqrtf(group_sum<TPR>(ss, lds) * inv + a.eps);
    const float mean = group_sum<TPR>(dot, lds) * inv;
    const float rx = POST ? 1.0f / sqrtf(group_sum<TPR>(xx, lds) * inv + a.eps) : 1.0f;
    float dot2 = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] += d[j] * y[j] * r;
      e[j] += r * (d[j] * w[j] - y[j] * (r * r) * mean);  // gradient of the total
      const float n = x[j] * rx, scaled = e[j] * sc[j];
      if (POST) {
        ds[j] += e[j] * n * pw[j];
        dp[j] += scaled * n;
        d[j] = scaled * pw[j];
        dot2 += d[j] * x[j];
      } else {
        ds[j] += e[j] * x[j];
        d[j] = scaled;
      }
    }
    store<RES, TPR>(static_cast<RES*>(a.dresidual) + flat, size, t, wide, e);
    if (POST) {
      const float m2 = group_sum<TPR>(dot2, lds) * inv;
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rx * (d[j] - x[j] * (rx * rx) * m2);
    }
    store<IO, TPR>(static_cast<IO*>(a.dx) + flat, size, t, wide, d);
  }
  float* dst = partial + int64_t(blockIdx.x) * 3 * a.size;
  if (a.dweight) write_partial<TPR>(dst, a.size, t, wide, dw, lds);
  if (a.dscale) write_partial<TPR>(dst + a.size, a.size, t, wide, ds, lds);
  if (POST && a.dpost_weight) write_partial<TPR>(dst + 2 * a.size, a.size, t, wide, dp, lds);
}

// out[set][e] = sum over the blocks of set `set` of partial[block][part][e], in order:
// blocks set, set + sets, ... of nblocks; 16 slices of the blocks per element.
struct SumArgs {
  const float* partial;
  float* out[3];
  int64_t size, pitch, nblocks, sets;
};

__global__ __launch_bounds__(1024) void partial_sum_kernel(SumArgs s) {
  __shared__ float lds[16][64];
  const int lane = int(threadIdx.x) & 63, slice = int(threadIdx.x) >> 6;
  const int64_t nb = (s.size + 63) / 64;
  const int64_t set = int64_t(blockIdx.x) / nb, e = int64_t(blockIdx.x) % nb * 64 + lane;
  const int part = int(blockIdx.y);
  if (!s.out[part]) return;
  const int64_t per_set = s.nblocks / s.sets;
  float x = 0.0f;
  if (e < s.size)
    for (int64_t k = slice; k < per_set; k += 16)
      x += s.partial[(set + k * s.sets) * s.pitch + part * s.size + e];
  lds[slice][lane] = x;
  __syncthreads();
  if (slice == 0 && e < s.size) {
#pragma unroll
    for (int k = 1; k < 16; ++k) x += lds[k][lane];
    s.out[part][set * s.size + e] = x;
  }
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads that hold one vector of this size: the smallest power of two (16 or more)
// whose eight elements each suffice.
int threads_of(int64_t size) {
  int t = 16;
  while (int64_t(t) * 8 < size) t *= 2;
  return t;
}

int64_t back_blocks(int64_t units, int64_t size, int64_t heads) {
  const int64_t groups = threads_of(size) < 256 ? 256 / threads_of(size) : 1;
  if (heads == 0) return 0;
  const int64_t most = kMaxBackBlocks > heads ? kMaxBackBlocks / heads : 1;
  const int64_t want = div_up(units, groups);
  return (want < most ? want : most) * heads;
}

bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename F>
hipError_t by_threads(int64_t size, F f) {
  switch (threads_of(size)) {
    case 16: f(std::integral_constant<int, 16>()); break;
    case 32: f(std::integral_constant<int, 32>()); break;
    case 64: f(std::integral_constant<int, 64>()); break;
    case 128: f(std::integral_constant<int, 128>()); break;
    case 256: f(std::integral_constant<int, 256>()); break;
    case 512: f(std::integral_constant<int, 512>()); break;
    default: f(std::integral_constant<int, 1024>()); break;  // size <= kNormMaxSize
  }
  return hipGetLastError();
}

// Whether a call's tensors allow 16-byte accesses throughout (one choice per call: the
// weights and the data share the threads' element order).
template <typename IO>
bool gated_wide(const GatedNormArgs& a) {
  const int64_t n = 16 / int64_t(sizeof(IO));
  return a.size % 8 == 0 && al16(a.x) && al16(a.z) && al16(a.out) && al16(a.dout) && al16(a.dx) && al16(a.dz) &&
         al16(a.weight) && a.xr % n == 0 && a.xh % n == 0 && a.zr % n == 0 && a.zh % n == 0;
}

bool add_wide(const AddNormArgs& a) {
  return a.size % 8 == 0 && al16(a.x) && al16(a.residual) && al16(a.out) && al16(a.residual_out) && al16(a.dout) &&
         al16(a.dresidual_out) && al16(a.dx) && al16(a.dresidual) && al16(a.weight) && al16(a.scale) &&
         al16(a.post_weight);
}

}  // namespace norm

using norm::bf16;

size_t gated_norm_bwd_workspace(int64_t rows, int64_t heads, int64_t size) {
  // whichever of the shared and the per-head weight needs more blocks
  const int64_t a = norm::back_blocks(rows * heads, size, 1), b = norm::back_blocks(rows, size, heads);
  return size_t(a > b ? a : b) * size_t(size) * 4;
}

size_t add_norm_bwd_workspace(int64_t rows, int64_t size) {
  return size_t(norm::back_blocks(rows, size, 1)) * 3 * size_t(size) * 4;
}

template <typename IO>
static hipError_t gated_fwd(const GatedNormArgs& a, hipStream_t stream) {
  return norm::by_threads(a.size, [&](auto tpr) {
    constexpr int T = decltype(tpr)::value, B = norm::threads<T>();
    int64_t n = norm::div_up(a.rows * a.heads, B / T);
    if (n > norm::kMaxBlocks) n = norm::kMaxBlocks;
    norm::gated_norm_kernel<IO, T><<<dim3(unsigned(n)), B, 0, stream>>>(a, norm::gated_wide<IO>(a));
  });
}

template <typename IO>
static hipError_t gated_bwd(const GatedNormArgs& a, float* ws, hipStream_t stream) {
  const int64_t sets = a.per_head ? a.heads : 1;
  const int64_t n = norm::back_blocks(a.per_head ? a.rows : a.rows * a.heads, a.size, sets);
  if (sets == 0) return hipSuccess;  // per-head weights of no heads
  // without rows there are no blocks, and the sums over none are zeros
  const hipError_t e = n == 0 ? hipSuccess : norm::by_threads(a.size, [&](auto tpr) {
    constexpr int T = decltype(tpr)::value, B = norm::threads<T>();
    norm::gated_norm_bwd_kernel<IO, T>
        <<<dim3(unsigned(n)), B, 0, stream>>>(a, ws, norm::gated_wide<IO>(a));
  });
  if (e != hipSuccess || !a.dweight) return e;
  const norm::SumArgs s{ws, {a.dweight, nullptr, nullptr}, a.size, a.size, n, sets};
  norm::partial_sum_kernel<<<dim3(unsigned(sets * norm::div_up(a.size, 64))), 1024, 0, stream>>>(s);
  return hipGetLastError();
}

template <typename IO, typename RES>
static hipError_t add_fwd(const AddNormArgs& a, hipStream_t stream) {
  return norm::by_threads(a.size, [&](auto tpr) {
    constexpr int T = decltype(tpr)::value, B = norm::threads<T>();
    int64_t n = norm::div_up(a.rows, B / T);
    if (n > norm::kMaxBlocks) n = norm::kMaxBlocks;
    norm::add_norm_kernel<IO, RES, T><<<dim3(unsigned(n)), B, 0, stream>>>(a, norm::add_wide(a));
  });
}

template <typename IO, typename RES>
static hipError_t add_bwd(const AddNormArgs& a, float* ws, hipStream_t stream) {
  const int64_t n = norm::back_blocks(a.rows, a.size, 1);
  const hipError_t e = n == 0 ? hipSuccess : norm::by_threads(a.size, [&](auto tpr) {
    constexpr int T = decltype(tpr)::value, B = norm::threads<T>();
    const dim3 grid{unsigned(n)};
    if (a.post_weight)
      norm::add_norm_bwd_kernel<IO, RES, T, true><<<grid, B, 0, stream>>>(a, ws, norm::add_wide(a));
    else
      norm::add_norm_bwd_kernel<IO, RES, T, false><<<grid, B, 0, stream>>>(a, ws, norm::add_wide(a));
  });
  if (e != hipSuccess || !(a.dweight || a.dscale || a.dpost_weight)) return e;
  const norm::SumArgs s{ws, {a.dweight, a.dscale, a.dpost_weight}, a.size, 3 * a.size, n, 1};
  norm::partial_sum_kernel<<<dim3(unsigned(norm::div_up(a.size, 64)), 3), 1024, 0, stream>>>(s);
  return hipGetLastError();
}

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream) {
  return a.io_bf16 ? gated_fwd<bf16>(a, stream) : gated_fwd<float>(a, stream);
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, float* ws, hipStream_t stream) {
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
