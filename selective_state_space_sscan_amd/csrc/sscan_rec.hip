// sscan_rec.hip -- the gated recurrence over whole sequences and for single tokens: one
// lane a channel, which walks its row token by token.
#include "sscan_rec_device.h"

namespace sscan {
namespace rec {

struct RowWalk {  // the tokens of a row in the order of the scan
  int64_t n, first, step;
  __device__ __forceinline__ RowWalk(const RecArgs& a, int64_t b) {
    n = a.len;
    if (a.lengths) n = a.lengths[b] < 0 ? 0 : a.lengths[b] < a.len ? a.lengths[b] : a.len;
    first = a.reverse ? n - 1 : 0;
    step = a.reverse ? -1 : 1;
  }
};

template <typename IO>
__device__ __forceinline__ float at(const RecIn& in, int64_t b, int64_t t, int64_t ch) {
  return float(static_cast<const IO*>(in.p)[b * in.b + t * in.t + ch]);
}

template <typename IO, bool GATED>
__global__ __launch_bounds__(64) void fwd_kernel(RecArgs a) {
  const int64_t ch = int64_t(blockIdx.x) * 64 + threadIdx.x, b = blockIdx.y;
  if (ch >= a.dim) return;
  const RowWalk row(a, b);
  const float rate = GATED ? decay_rate(a.lam, ch, a.c) : 0.0f;
  float h = a.h0 ? a.h0[b * a.dim + ch] : 0.0f;
  IO* out = static_cast<IO*>(a.out) + b * a.len * a.dim + ch;
  for (int64_t k = 0; k < row.n; ++k) {
    const int64_t t = row.first + k * row.step;
    const Decay d = decay<GATED>(at<IO>(a.g, b, t, ch), rate);
    float u = at<IO>(a.x, b, t, ch) * d.w;
    if (a.i.p) u *= sigmoid(at<IO>(a.i, b, t, ch));
    h = fmaf(d.a, h, u);
    float y = h;
    if (a.z.p) {
      const float z = at<IO>(a.z, b, t, ch);
      y *= z * sigmoid(z);
    }
    out[t * a.dim] = IO(y);
  }
  for (int64_t t = row.n; t < a.len; ++t) out[t * a.dim] = IO(0.0f);
  a.h_last[b * a.dim + ch] = h;
}

template <typename IO>
hipError_t fwd(const RecArgs& a, hipStream_t stream) {
  const dim3 grid(unsigned((a.dim + 63) / 64), unsigned(a.batch));
  if (a.lam)
    fwd_kernel<IO, true><<<grid, 64, 0, stream>>>(a);
  else
    fwd_kernel<IO, false><<<grid, 64, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace rec

size_t rec_workspace(int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_rec_fwd(const RecArgs& a, char*, hipStream_t stream) {
  if (a.kept.x && a.len > 0) {
    const RecIn in[4] = {a.x, a.g, a.i, a.z};
    int8_t* q[4] = {a.kept.x, a.kept.g, a.kept.i, a.kept.z};
    float* s[4] = {a.kept.xs, a.kept.gs, a.kept.is, a.kept.zs};
    for (int k = 0; k < 4; ++k) {
      if (!in[k].p) continue;
      const hipError_t e = launch_pack8({in[k].p, in[k].b, in[k].t, q[k], s[k], nullptr, a.batch, a.len, a.dim, a.io_bf16},
                                        stream);
      if (e != hipSuccess) return e;
    }
  }
  return a.io_bf16 ? rec::fwd<rec::bf16>(a, stream) : rec::fwd<float>(a, stream);
}

hipError_t launch_rec_step(const RecArgs& a, hipStream_t stream) { return launch_rec_fwd(a, nullptr, stream); }

}  // namespace sscan
