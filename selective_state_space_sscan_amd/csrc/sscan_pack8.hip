// sscan_pack8.hip -- activations in 8 bits: blocks of 64 elements of a row, each with the
// scale max|x| / 127.  Eight lanes take a block, eight elements a lane, by 16-byte accesses
// at whatever alignment the rows have.  Bound by memory: 16384 x 1536 bf16 there and back 30
// us (5.2 TB/s; the tensors fit the last cache); one element a lane took 128.
#include "sscan_pack8.h"

#include "sscan_norm_device.h"

namespace sscan {
namespace rec {

// The walk of eight lanes over the units (row, block of 64): row and block by division once,
// then by the step's quotient and remainder.
constexpr int kUnits = 256 / 8, kMaxGrid = 8192;

struct UnitWalk {
  int64_t u, row, k, units, blocks, step, step_rows, step_k;
  __device__ __forceinline__ UnitWalk(int64_t rows, int64_t blocks_) : blocks(blocks_) {
    units = rows * blocks;
    u = int64_t(blockIdx.x) * kUnits + threadIdx.x / 8;
    row = u / blocks;
    k = u % blocks;
    step = int64_t(gridDim.x) * kUnits;
    step_rows = step / blocks;
    step_k = step % blocks;
  }
  __device__ __forceinline__ void next() {
    u += step;
    row += step_rows;
    k += step_k;
    if (k >= blocks) {
      k -= blocks;
      ++row;
    }
  }
};

typedef int8_t i8x8 __attribute__((ext_vector_type(8), aligned(1)));

template <typename IO>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs a, int64_t blocks) {
  const int sub = int(threadIdx.x) % 8;
  for (UnitWalk w(a.rows, blocks); w.u < w.units; w.next()) {
    const int64_t e = w.k * kPackBlock + sub * 8;
    const int n = e + 8 <= a.size ? 8 : e < a.size ? int(a.size - e) : 0;
    const IO* p = static_cast<const IO*>(a.x) + w.row * a.x_stride + e;
    float x[8];
    if (n == 8) {
      const auto v = norm::load_eight(p);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = float(v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = j < n ? float(p[j]) : 0.0f;
    }
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, magnitude(x[j]));
#pragma unroll
    for (int s = 1; s < 8; s *= 2) m = max(m, unsigned(__shfl_xor(int(m), s)));
    const Scale scale(m);
    i8x8 q;
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = int8_t(scale.steps(x[j]));
    int8_t* to = a.q + w.row * a.size + e;
    if (n == 8) {
      *reinterpret_cast<i8x8*>(to) = q;
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) to[j] = q[j];
    }
    if (sub == 0) a.scale[w.row * blocks + w.k] = scale.step;
  }
}

template <typename IO>
__global__ __launch_bounds__(256) void unpack_kernel(PackArgs a, int64_t blocks) {
  const int sub = int(threadIdx.x) % 8;
  for (UnitWalk w(a.rows, blocks); w.u < w.units; w.next()) {
    const int64_t e = w.k * kPackBlock + sub * 8;
    const int n = e + 8 <= a.size ? 8 : e < a.size ? int(a.size - e) : 0;
    const float scale = a.scale[w.row * blocks + w.k];
    const int8_t* from = a.q + w.row * a.size + e;
    IO* to = static_cast<IO*>(a.out) + w.row * a.size + e;
    if (n == 8) {
      const i8x8 q = *reinterpret_cast<const i8x8*>(from);
      typename delta::Io<IO>::V8 y;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = IO(float(q[j]) * scale);
      norm::store_eight(to, y);
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) to[j] = IO(float(from[j]) * scale);
    }
  }
}

}  // namespace rec

static dim3 pack_grid(int64_t units) {
  const int64_t n = (units + rec::kUnits - 1) / rec::kUnits;
  return dim3(unsigned(n < rec::kMaxGrid ? n : rec::kMaxGrid));
}

hipError_t launch_pack8(const PackArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.size + kPackBlock - 1) / kPackBlock;
  if (a.io_bf16)
    rec::pack_kernel<rec::bf16><<<pack_grid(a.rows * blocks), 256, 0, stream>>>(a, blocks);
  else
    rec::pack_kernel<float><<<pack_grid(a.rows * blocks), 256, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

hipError_t launch_unpack8(const PackArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.size + kPackBlock - 1) / kPackBlock;
  if (a.io_bf16)
    rec::unpack_kernel<rec::bf16><<<pack_grid(a.rows * blocks), 256, 0, stream>>>(a, blocks);
  else
    rec::unpack_kernel<float><<<pack_grid(a.rows * blocks), 256, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace sscan
