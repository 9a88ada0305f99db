// sscan_layer_norm.hip -- layer norm fused with the residual sum in front of it, and its
// gradients.  Rows are held in registers as in the RMS norms (sscan_norm_device.h): every
// input is read once and every output written once.  Mean and variance are by two rounds of
// sums in float32 over registers.  Bound by HBM: 16384 x 1536 bf16 with a float32 residual take
// 57 us, where a large copy would move their bytes in 59 (part stays in the last cache), their
// gradients 85, sum over blocks included (79); 8192 x 4096 71 (79) and 117 (105).
#include "sscan_norm_device.h"
#include "sscan_rec.h"

namespace sscan {
namespace norm {

constexpr int kMaxLayerBlocks = 8192, kMaxLayerBackBlocks = 1024;

// The mean of the squares around a mean that is off by `off`.  The mean is the quotient of a
// rounded sum, off by up to 17 U of the values' size (U = 2^-24), which rows of nearly equal
// values would show as a deviation: so the deviations' own mean is summed along with their
// squares and taken out.  Rows of one value then have none at all: their deviations are the
// same few steps, whose sum and quotient are exact.  The sum more costs 1% to 2% up to sizes of
// 4096, in rows of 8192, which a block of 1024 threads holds, 4% and 5% (2048 x 8192 f32 46.1 ->
// 47.9 us, gradients 80.6 -> 84.9).
// The product is not rounded by itself: squares beyond float32 stay an infinity.
__device__ __forceinline__ float variance(float squares, float off) { return fmaxf(fmaf(-off, off, squares), 0.0f); }

// total = residual + x (stored as RES where wanted), out = (total - mean) / sqrt(var + eps) * weight + bias
template <typename IO, typename RES, int TPR, bool whole>
__global__ __launch_bounds__(threads<TPR>()) void layer_norm_kernel(LayerNormArgs a) {
  __shared__ float lds[2][3][16];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  const int64_t step = int64_t(gridDim.x) * kGroups;
  const Place at = place<whole>(int(a.size), t);
  float w[8], c[8], next_x[8], next_y[8];
  const auto load_next = [&](int64_t u) {
    const int size = u < a.rows ? int(a.size) : 0;
    load<whole>(static_cast<const IO*>(a.x) + (size ? u * a.x_stride : 0), size, t, next_x);
    load<whole>(static_cast<const RES*>(a.residual) + (size ? u * a.size : 0), a.residual ? size : 0, t, next_y);
  };
  load_next(int64_t(blockIdx.x) * kGroups + grp);
  load_or<whole>(a.weight, int(a.size), t, 1.0f, w);
  load_or<whole>(a.bias, int(a.size), t, 0.0f, c);
  const float inv = 1.0f / float(a.size);
  int turn = 0;
  for (int64_t u0 = int64_t(blockIdx.x) * kGroups; u0 < a.rows; u0 += step) {
    const int64_t u = u0 + grp, flat = u * a.size;
    const int size = u < a.rows ? int(a.size) : 0;
    float x[8], sum[1] = {0.0f}, dev[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = next_y[j] + next_x[j];
      if (a.total) x[j] = float(RES(x[j]));
      sum[0] += x[j];
    }
    load_next(u + step);
    if (a.total) store<whole>(static_cast<RES*>(a.total) + flat, size, t, x);
    group_sum<TPR>(sum, lds, turn);
    turn ^= 1;
    const float mean = sum[0] / float(a.size);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // places that hold no element of their own count for nothing
      x[j] = j >= at.dup && at.off + j < size ? x[j] - mean : 0.0f;
      dev[0] += x[j];
      dev[1] += x[j] * x[j];
    }
    group_sum<TPR>(dev, lds, turn);
    turn ^= 1;
    const float off = dev[0] / float(a.size), r = 1.0f / sqrtf(variance(dev[1] * inv, off) + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (x[j] - off) * r * w[j] + c[j];
    store<whole>(static_cast<IO*>(a.out) + flat, size, t, x);
  }
}

// With n = (x - mean) r and dn = dout w the gradient at x is r (dn - mean(dn) - n mean(dn n)).
template <typename IO, typename RES, int TPR, bool whole>
__global__ __launch_bounds__(threads<TPR>()) void layer_norm_bwd_kernel(LayerNormArgs a, float* partial) {
  __shared__ float lds[2][3][16];
  __shared__ float sums[partial_lds<TPR>()];
  constexpr int kGroups = threads<TPR>() / TPR;
  const int t = int(threadIdx.x) % TPR, grp = int(threadIdx.x) / TPR;
  const int64_t step = int64_t(gridDim.x) * kGroups;
  const Place at = place<whole>(int(a.size), t);
  float w[8], dw[8] = {}, db[8] = {}, next_x[8], next_d[8], next_e[8];
  const auto load_next = [&](int64_t u) {
    const int size = u < a.rows ? int(a.size) : 0;
    const int64_t flat = size ? u * a.size : 0;
    load<whole>(static_cast<const RES*>(a.x) + (size ? u * a.x_stride : 0), size, t, next_x);
    load<whole>(static_cast<const IO*>(a.dout) + flat, size, t, next_d);
    load<whole>(static_cast<const RES*>(a.dtotal) + flat, a.dtotal ? size : 0, t, next_e);
  };
  load_next(int64_t(blockIdx.x) * kGroups + grp);
  load_or<whole>(a.weight, int(a.size), t, 1.0f, w);
  const float inv = 1.0f / float(a.size);
  int turn = 0;
  for (int64_t u0 = int64_t(blockIdx.x) * kGroups; u0 < a.rows; u0 += step) {
    const int64_t u = u0 + grp, flat = u * a.size;
    const int size = u < a.rows ? int(a.size) : 0;
    float x[8], d[8], e[8], sum[2] = {0.0f, 0.0f}, dev[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = next_x[j];
      d[j] = next_d[j];
      e[j] = next_e[j];
      sum[0] += x[j];
      sum[1] += d[j] * w[j];
    }
    load_next(u + step);
    group_sum<TPR>(sum, lds, turn);
    turn ^= 1;
    const float mean = sum[0] / float(a.size), dmean = sum[1] * inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = j >= at.dup && at.off + j < size ? x[j] - mean : 0.0f;
      dev[0] += x[j];
      dev[1] += x[j] * x[j];
      dev[2] += d[j] * w[j] * x[j];
    }
    group_sum<TPR>(dev, lds, turn);
    turn ^= 1;
    // a group past the last row holds zeros, and leaves the sums alone where eps is 0 too
    const float off = dev[0] / float(a.size), var = variance(dev[1] * inv, off);
    const float r = kGroups > 1 && !size ? 0.0f : 1.0f / sqrtf(var + a.eps), dot = (dev[2] * inv - off * dmean) * r;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = (x[j] - off) * r;
      dw[j] += d[j] * x[j];
      db[j] += d[j];
      e[j] += r * (d[j] * w[j] - dmean - x[j] * dot);
    }
    store<whole>(static_cast<IO*>(a.dx) + flat, size, t, e);
    if (a.dresidual) store<whole>(static_cast<RES*>(a.dresidual) + flat, size, t, e);
  }
  float* dst = partial + int64_t(blockIdx.x) * 2 * a.size;
  if (a.dweight) write_partial<TPR, whole>(dst, int(a.size), t, dw, sums);
  if (a.dbias) write_partial<TPR, whole>(dst + a.size, int(a.size), t, db, sums);
}

static int64_t layer_back_blocks(int64_t rows, int64_t size) {
  const int64_t groups = threads_of(size) < 256 ? 256 / threads_of(size) : 1, n = div_up(rows, groups);
  return n < kMaxLayerBackBlocks ? n : kMaxLayerBackBlocks;
}

template <typename IO, typename RES>
static hipError_t layer_fwd(const LayerNormArgs& a, hipStream_t stream) {
  return by_shape(a.size, [&](auto tpr, auto whole) {
    constexpr int T = decltype(tpr)::value, B = threads<T>();
    int64_t n = div_up(a.rows, B / T);
    if (n > kMaxLayerBlocks) n = kMaxLayerBlocks;
    layer_norm_kernel<IO, RES, T, decltype(whole)::value><<<dim3(unsigned(n)), B, 0, stream>>>(a);
  });
}

template <typename IO, typename RES>
static hipError_t layer_bwd(const LayerNormArgs& a, float* ws, hipStream_t stream) {
  const int64_t n = layer_back_blocks(a.rows, a.size);
  const hipError_t e = n == 0 ? hipSuccess : by_shape(a.size, [&](auto tpr, auto whole) {
    constexpr int T = decltype(tpr)::value, B = threads<T>();
    layer_norm_bwd_kernel<IO, RES, T, decltype(whole)::value><<<dim3(unsigned(n)), B, 0, stream>>>(a, ws);
  });
  if (e != hipSuccess || !(a.dweight || a.dbias)) return e;
  float* const out[2] = {a.dweight, a.dbias};
  return launch_row_sums(ws, out, 2, a.size, n, stream);
}

}  // namespace norm

size_t layer_norm_bwd_workspace(int64_t rows, int64_t size) {
  return size_t(norm::layer_back_blocks(rows, size)) * 2 * size_t(size) * 4;
}

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t stream) {
  using norm::bf16;
  if (a.io_bf16) return a.res_bf16 ? norm::layer_fwd<bf16, bf16>(a, stream) : norm::layer_fwd<bf16, float>(a, stream);
  return a.res_bf16 ? norm::layer_fwd<float, bf16>(a, stream) : norm::layer_fwd<float, float>(a, stream);
}

hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, float* ws, hipStream_t stream) {
  using norm::bf16;
  if (a.io_bf16) return a.res_bf16 ? norm::layer_bwd<bf16, bf16>(a, ws, stream) : norm::layer_bwd<bf16, float>(a, ws, stream);
  return a.res_bf16 ? norm::layer_bwd<float, bf16>(a, ws, stream) : norm::layer_bwd<float, float>(a, ws, stream);
}

}  // namespace sscan
