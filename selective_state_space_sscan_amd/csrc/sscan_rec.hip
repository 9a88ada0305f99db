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
    return *reinterpret_cast<const V*>(static_cast<const IO*>(in.p) + b * in.b + ch);
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
      const Decay d = decay<GATED>(part<V, C>(g, c), GATED ? decay_rate(a.lam, ch + c, a.c) : 0.0f);
      float u = part<V, C>(x, c) * d.w;
      if (a.i.p) u *= sigmoid(part<V, C>(i, c));
      y[c] = fmaf(d.a, state[c], u);
      state[c] = y[c];
      if (a.z.p) {
        const float q = part<V, C>(z, c);
        y[c] *= q * sigmoid(q);
      }
    }
  }
  *reinterpret_cast<V*>(static_cast<IO*>(a.out) + b * a.dim + ch) = packed<IO, C>(y);
}

// The state handed through where there are no tokens.
__global__ __launch_bounds__(256) void pass_kernel(const float* from, float* to, int64_t n) {
  const int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (k < n) to[k] = from ? from[k] : 0.0f;
}

constexpr int kT = 16;               // tokens of a wave's tile
constexpr int kWaves = 8;            // of a block where rows have several segments

int channels_of(int64_t dim) { return dim % 2 == 0 ? 2 : 1; }

struct Plan {
  int c, waves;
  int64_t groups, nseg, words;       // bytes of the maps and states
};

Plan plan_of(int64_t batch, int64_t len, int64_t dim) {
  Plan p;
  p.c = channels_of(dim);
  p.groups = up(dim, 64 * p.c);
  const int64_t tiles = up(len, kT);
  p.waves = tiles <= kMaxWaves ? int(tiles) : kWaves;
  p.nseg = tiles <= kMaxWaves ? 1 : up(tiles, p.waves);
  p.words = p.nseg > 1 ? (p.nseg + p.nseg / kRun) * batch * p.groups * 64 * p.c * 8 : 0;
  return p;
}

template <typename IO, int C>
hipError_t fwd(const RecArgs& a, const Plan& plan, char* workspace, hipStream_t stream) {
  uint64_t* words = reinterpret_cast<uint64_t*>(workspace + 256);
  const TileArgs p{a, words, words + plan.nseg * a.batch * plan.groups * 64 * C, reinterpret_cast<unsigned*>(workspace),
                   nullptr, int(plan.nseg), unsigned(plan.groups)};
  const dim3 grid(unsigned(plan.nseg * a.batch * plan.groups)), block(unsigned(plan.waves * 64));
  const size_t lds = size_t(plan.waves) * 2 * 64 * C * 4;
  if (plan.nseg > 1) {
    const int64_t n = plan.words / 16, blocks = up(n, 256 * 4);
    clear_kernel<<<dim3(unsigned(blocks < 2048 ? blocks : 2048)), 256, 0, stream>>>(reinterpret_cast<uint4*>(words), n, p.ticket);
  }
  by_flag(a.lam != nullptr, [&](auto gated) {
    by_flag(a.i.p != nullptr, [&](auto igate) {
      by_flag(a.z.p != nullptr, [&](auto zgate) {
        by_flag(plan.nseg > 1, [&](auto split) {
          fwd_kernel<IO, C, kT, decltype(gated)::value, decltype(igate)::value, decltype(zgate)::value,
                     decltype(split)::value, true, false><<<grid, block, lds, stream>>>(p);
        });
      });
    });
  });
  return hipGetLastError();
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

size_t rec_workspace(int64_t batch, int64_t len, int64_t dim, bool) {
  const rec::Plan p = rec::plan_of(batch, len, dim);
  return p.nseg > 1 ? size_t(p.words) + 256 : 0;
}

hipError_t launch_rec_fwd(const RecArgs& a, char* workspace, hipStream_t stream) {
  if (a.len == 0) {
    const int64_t n = a.batch * a.dim;
    rec::pass_kernel<<<dim3(unsigned(rec::up(n, 256))), 256, 0, stream>>>(a.h0, a.h_last, n);
    return hipGetLastError();
  }
  if (a.kept.x) {
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
  const rec::Plan p = rec::plan_of(a.batch, a.len, a.dim);
  if (a.io_bf16)
    return p.c == 2 ? rec::fwd<rec::bf16, 2>(a, p, workspace, stream) : rec::fwd<rec::bf16, 1>(a, p, workspace, stream);
  return p.c == 2 ? rec::fwd<float, 2>(a, p, workspace, stream) : rec::fwd<float, 1>(a, p, workspace, stream);
}

hipError_t launch_rec_step(const RecArgs& a, hipStream_t stream) {
  const int c = rec::channels_of(a.dim);
  if (a.io_bf16) return c == 2 ? rec::step<rec::bf16, 2>(a, stream) : rec::step<rec::bf16, 1>(a, stream);
  return c == 2 ? rec::step<float, 2>(a, stream) : rec::step<float, 1>(a, stream);
}

}  // namespace sscan
