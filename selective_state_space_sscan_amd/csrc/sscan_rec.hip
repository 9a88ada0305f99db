// sscan_rec.hip -- the gated recurrence over whole sequences and for single tokens.
#include "sscan_rec_fwd.h"

namespace sscan {
namespace rec {

// One token from a stored state.
template <typename IO, int C, bool GATED>
__global__ __launch_bounds__(64) void step_kernel(RecArgs a) {
  typedef typename Vec<IO, C>::V V;
  const unsigned groups = unsigned((a.dim + 64 * C - 1) / (64 * C));
  const int64_t ch = (int64_t(blockIdx.x % groups) * 64 + threadIdx.x) * C, b = blockIdx.x / groups;
  if (ch >= a.dim) return;
  const auto load = [&](const RecIn& in) {
    return load_any<IO, C>(static_cast<const IO*>(in.p) + b * in.b + ch);
  };
  float* state = a.h_last + b * a.dim + ch;
  const bool live = !a.lengths || a.lengths[b] > 0;
  float y[C];
#pragma unroll
  for (int c = 0; c < C; ++c) y[c] = 0.0f;
  if (live) {
    const V x = load(a.x), g = load(a.g), i = a.i.p ? load(a.i) : V{}, z = a.z.p ? load(a.z) : V{};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Decay d = decay<GATED>(part<C>(g, c), GATED ? decay_rate(a.lam, ch + c, a.c) : 0.0f, true);
      float u = part<C>(x, c) * d.w;
      if (a.i.p) u *= sigmoid(part<C>(i, c));
      y[c] = fmaf(d.a, state[c], u);
      state[c] = y[c];
      if (a.z.p) {
        const float q = part<C>(z, c);
        y[c] *= q * sigmoid(q);
      }
    }
  }
  store_any<IO, C>(static_cast<IO*>(a.out) + b * a.dim + ch, packed<IO, C>(y));
}

// The state handed through where there are no tokens.
__global__ __launch_bounds__(256) void pass_kernel(const float* from, float* to, int64_t n) {
  const int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (k < n) to[k] = from ? from[k] : 0.0f;
}

template <typename IO, int C>
hipError_t step(const RecArgs& a, hipStream_t stream) {
  const dim3 grid(unsigned(up(a.dim, 64 * C) * a.batch));
  if (a.lam)
    step_kernel<IO, C, true><<<grid, 64, 0, stream>>>(a);
  else
    step_kernel<IO, C, false><<<grid, 64, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace rec

size_t rec_workspace(int64_t batch, int64_t len, int64_t dim, bool io_bf16) {
  const rec::Plan p = rec::plan_of(batch, len, dim, io_bf16);
  return p.words ? size_t(p.words) + 256 : 0;
}

hipError_t launch_rec_fwd(const RecArgs& a, char* workspace, hipStream_t stream) {
  if (a.len == 0) {
    const int64_t n = a.batch * a.dim;
    rec::pass_kernel<<<dim3(unsigned(rec::up(n, 256))), 256, 0, stream>>>(a.h0, a.h_last, n);
    return hipGetLastError();
  }
  const rec::Plan p = rec::plan_of(a.batch, a.len, a.dim, a.io_bf16);
  if (a.kept.x) return rec::launch_keep(a, p, workspace, stream);
  return rec::by_lane(p.c, a.io_bf16, [&](auto io, auto c) {
    return rec::fwd<decltype(io), decltype(c)::value, false>(a, p, workspace, stream);
  });
}

hipError_t launch_rec_step(const RecArgs& a, hipStream_t stream) {
  return rec::by_lane(rec::channels_of(a.dim), a.io_bf16, [&](auto io, auto c) {
    return rec::step<decltype(io), decltype(c)::value>(a, stream);
  });
}

}  // namespace sscan
