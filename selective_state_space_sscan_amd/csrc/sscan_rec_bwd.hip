// sscan_rec_bwd.hip -- gradients of the gated recurrence: one lane a channel, which walks its
// row forwards, keeping the state before each token, and then back.
#include "sscan_rec_device.h"

namespace sscan {
namespace rec {

template <typename IO>
struct Source {  // an input, or what its 8 bits stand for
  const IO* p;
  const int8_t* q;
  const float* scale;
  int64_t tstride, dim, blocks, ch;
  __device__ __forceinline__ Source(const RecIn& in, const int8_t* q_, const float* s_, const RecArgs& a, int64_t b,
                                    int64_t ch_)
      : p(in.p ? static_cast<const IO*>(in.p) + b * in.b + ch_ : nullptr), q(q_), scale(s_), tstride(in.t), dim(a.dim),
        blocks((a.dim + kPackBlock - 1) / kPackBlock), ch(ch_) {
    if (q) {
      q += b * a.len * dim + ch;
      scale += b * a.len * blocks + ch / kPackBlock;
    }
  }
  __device__ __forceinline__ bool given() const { return p || q; }
  __device__ __forceinline__ float at(int64_t t) const {
    return q ? float(q[t * dim]) * scale[t * blocks] : float(p[t * tstride]);
  }
};

template <typename IO, bool GATED>
__global__ __launch_bounds__(64) void bwd_kernel(RecBwdArgs w, float* states, float* partial) {
  const RecArgs& a = w.f;
  const int64_t ch = int64_t(blockIdx.x) * 64 + threadIdx.x, b = blockIdx.y;
  if (ch >= a.dim) return;
  int64_t n = a.len;
  if (a.lengths) n = a.lengths[b] < 0 ? 0 : a.lengths[b] < a.len ? a.lengths[b] : a.len;
  const int64_t first = a.reverse ? n - 1 : 0, step = a.reverse ? -1 : 1;
  const Source<IO> sx(a.x, a.kept.x, a.kept.xs, a, b, ch), sg(a.g, a.kept.g, a.kept.gs, a, b, ch),
      si(a.i, a.kept.i, a.kept.is, a, b, ch), sz(a.z, a.kept.z, a.kept.zs, a, b, ch);
  const float rate = GATED ? decay_rate(a.lam, ch, a.c) : 0.0f;
  const int64_t base = b * a.len * a.dim + ch;
  float h = a.h0 ? a.h0[b * a.dim + ch] : 0.0f;
  for (int64_t k = 0; k < n; ++k) {
    const int64_t t = first + k * step;
    states[base + t * a.dim] = h;
    const Decay d = decay<GATED>(sg.at(t), rate);
    h = fmaf(d.a, h, sx.at(t) * d.w * (si.given() ? sigmoid(si.at(t)) : 1.0f));
  }
  float carry = w.dh_last ? w.dh_last[b * a.dim + ch] : 0.0f, dlam = 0.0f;
  const IO* dout = static_cast<const IO*>(w.dout) + base;
  IO *dx = static_cast<IO*>(w.dx) + base, *dg = static_cast<IO*>(w.dg) + base, *di = static_cast<IO*>(w.di) + base,
     *dz = static_cast<IO*>(w.dz) + base;
  for (int64_t k = n - 1; k >= 0; --k) {
    const int64_t t = first + k * step, e = t * a.dim;
    const Decay d = decay<GATED>(sg.at(t), rate);
    const float x = sx.at(t), s = si.given() ? sigmoid(si.at(t)) : 1.0f, before = states[base + e];
    float back = float(dout[e]);
    if (sz.given()) {
      const float z = sz.at(t), q = sigmoid(z);
      dz[e] = IO(back * fmaf(d.a, before, x * d.w * s) * q * (1.0f + z * (1.0f - q)));
      back *= z * q;
    }
    const float adj = back + carry, slope = d.w > 0.0f ? d.a * d.a * __builtin_amdgcn_rcpf(d.w) : 0.0f;
    carry = d.a * adj;
    float dlog = carry * before;
    if (GATED) {
      dlog -= adj * s * x * slope;
      dg[e] = IO(-dlog * rate * d.r * (1.0f - d.r));
      dlam -= dlog * d.r;
    } else {
      dg[e] = IO(dlog);
    }
    dx[e] = IO(adj * d.w * s);
    if (si.given()) di[e] = IO(adj * d.w * x * s * (1.0f - s));
  }
  for (int64_t t = n; t < a.len; ++t) {
    const int64_t e = t * a.dim;
    dx[e] = dg[e] = IO(0.0f);
    if (si.given()) di[e] = IO(0.0f);
    if (sz.given()) dz[e] = IO(0.0f);
  }
  if (w.dh0) w.dh0[b * a.dim + ch] = carry;
  if (GATED && w.dlam) partial[b * a.dim + ch] = dlam * a.c / (1.0f + expf(-a.lam[ch]));
}

template <typename IO>
hipError_t bwd(const RecBwdArgs& w, char* workspace, hipStream_t stream) {
  const RecArgs& a = w.f;
  const dim3 grid(unsigned((a.dim + 63) / 64), unsigned(a.batch));
  float* states = reinterpret_cast<float*>(workspace);
  float* partial = states + a.batch * a.len * a.dim;
  if (a.batch == 0)
    ;  // the sum over no rows is zeros
  else if (a.lam)
    bwd_kernel<IO, true><<<grid, 64, 0, stream>>>(w, states, partial);
  else
    bwd_kernel<IO, false><<<grid, 64, 0, stream>>>(w, states, partial);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !w.dlam) return e;
  float* const out[1] = {w.dlam};
  return launch_row_sums(partial, out, 1, a.dim, a.batch, stream);
}

}  // namespace rec

size_t rec_bwd_workspace(int64_t batch, int64_t len, int64_t dim, bool) {
  return size_t(batch) * size_t(len + 1) * size_t(dim) * 4;
}

hipError_t launch_rec_bwd(const RecBwdArgs& a, char* workspace, hipStream_t stream) {
  return a.f.io_bf16 ? rec::bwd<rec::bf16>(a, workspace, stream) : rec::bwd<float>(a, workspace, stream);
}

}  // namespace sscan
