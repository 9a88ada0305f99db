// sscan_pack8.hip -- activations in 8 bits: blocks of 64 elements of a row, each with the
// scale max|x| / 127.  One wave a block.
#include "sscan_rec_device.h"

namespace sscan {
namespace rec {

constexpr float kTiny = 0x1p-100f;

template <typename IO>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs a, int64_t blocks) {
  const int64_t unit = int64_t(blockIdx.x) * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
  if (unit >= a.batch * a.rows * blocks) return;
  const int64_t flat = unit / blocks, k = unit % blocks, e = k * kPackBlock + lane;
  const int64_t b = flat / a.rows, r = flat % a.rows;
  const float x = e < a.size ? float(static_cast<const IO*>(a.x)[b * a.xb + r * a.xr + e]) : 0.0f;
  // as whole numbers, so that a NaN is the largest
  unsigned m = __float_as_uint(x) & 0x7fffffffu;
#pragma unroll
  for (int s = 1; s < 64; s *= 2) m = max(m, unsigned(__shfl_xor(int(m), s)));
  const float top = __uint_as_float(m);
  const bool bad = m >= 0x7f800000u, none = top < kTiny;
  const float y = bad || none ? 0.0f : x * (127.0f / top);
  if (e < a.size) a.q[flat * a.size + e] = int8_t(rintf(y));
  if (lane == 0) a.scale[flat * blocks + k] = bad ? __uint_as_float(0x7fc00000u) : none ? 0.0f : top / 127.0f;
}

template <typename IO>
__global__ __launch_bounds__(256) void unpack_kernel(PackArgs a, int64_t blocks) {
  const int64_t unit = int64_t(blockIdx.x) * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
  if (unit >= a.batch * a.rows * blocks) return;
  const int64_t flat = unit / blocks, k = unit % blocks, e = k * kPackBlock + lane;
  if (e < a.size) static_cast<IO*>(a.out)[flat * a.size + e] = IO(float(a.q[flat * a.size + e]) * a.scale[flat * blocks + k]);
}

}  // namespace rec

hipError_t launch_pack8(const PackArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.size + kPackBlock - 1) / kPackBlock;
  const dim3 grid(unsigned((a.batch * a.rows * blocks + 3) / 4));
  if (a.io_bf16)
    rec::pack_kernel<rec::bf16><<<grid, 256, 0, stream>>>(a, blocks);
  else
    rec::pack_kernel<float><<<grid, 256, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

hipError_t launch_unpack8(const PackArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.size + kPackBlock - 1) / kPackBlock;
  const dim3 grid(unsigned((a.batch * a.rows * blocks + 3) / 4));
  if (a.io_bf16)
    rec::unpack_kernel<rec::bf16><<<grid, 256, 0, stream>>>(a, blocks);
  else
    rec::unpack_kernel<float><<<grid, 256, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace sscan
