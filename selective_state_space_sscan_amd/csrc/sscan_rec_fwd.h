// sscan_rec_fwd.h -- the recurrence over a segment of a row: the forward's kernel, and that of
// the states between segments, which the backward pass starts from.
#pragma once

#include "sscan_rec_tile.h"

namespace sscan {
namespace rec {

// One segment a block (sscan_rec_tile.h).  A lane first turns its tokens into decays and
// inputs, which it holds in registers with their map; the waves' maps meet in LDS, wave 0
// finds the state that enters the segment (from the row's segments before, where there are
// any) and from it those that enter the waves, and every wave walks its tokens once more,
// now from its state, and answers.  SPLIT: rows have several segments.  OUT: outputs are
// wanted, not the states between segments alone (whose last segment has no block).  KEPT:
// the inputs come in 8 bits.
template <typename IO, int C, int T, bool GATED, bool IGATE, bool ZGATE, bool SPLIT, bool OUT, bool KEPT>
__global__ __launch_bounds__(kMaxWaves * 64) void fwd_kernel(TileArgs p) {
  typedef typename Vec<IO, C>::V V;
  extern __shared__ float lds[];     // [waves][2][64 C]: A and H; then the waves' entry states in A's place
  __shared__ unsigned number;
  const RecArgs& a = p.a;
  const int lane = int(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int waves = int(blockDim.x) >> 6;
  const Tile tile = Tile::of<SPLIT>(p, &number);
  const int seg = tile.seg;
  const int64_t b = tile.b, group = tile.group;
  const int64_t ch = (group * 64 + lane) * C;
  const bool on = ch < a.dim;
  const int64_t at = on ? ch : 0;    // lanes beyond the last channel read the first ones
  const Span span(a, b, (int64_t(seg) * waves + wave) * T, T);

  float rate[C];
#pragma unroll
  for (int c = 0; c < C; ++c) rate[c] = GATED ? decay_rate(a.lam, at + c, a.c) : 0.0f;

  const auto load = [&](const RecIn& in, const int8_t* q, const float* s, In<IO, C, KEPT>(&v)[T]) {
#pragma unroll
    for (int j = 0; j < T; ++j) v[j].load(a, in, q, s, b, span.place(j < span.live ? j : span.live - 1), at);
  };
  float A[T][C], U[T][C];
  In<IO, C, KEPT> z[T];
  if (span.live > 0) {
    In<IO, C, KEPT> x[T], g[T], i[T];
    load(a.x, a.kept.x, a.kept.xs, x);
    load(a.g, a.kept.g, a.kept.gs, g);
    if (IGATE) load(a.i, a.kept.i, a.kept.is, i);
    if (OUT && ZGATE) load(a.z, a.kept.z, a.kept.zs, z);
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const Decay d = decay<GATED>(g[j].get(c), rate[c]);
        float u = x[j].get(c) * d.w;
        if (IGATE) u *= sigmoid(i[j].get(c));
        const bool live = j < span.live;
        A[j][c] = live ? d.a : 1.0f;
        U[j][c] = live ? u : 0.0f;
      }
  } else {
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        A[j][c] = 1.0f;
        U[j][c] = 0.0f;
      }
  }
  float* mine = lds + wave * (2 * 64 * C) + lane;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float P = A[0][c], H = U[0][c];
#pragma unroll
    for (int j = 1; j < T; ++j) {
      P *= A[j][c];
      H = fmaf(A[j][c], H, U[j][c]);
    }
    mine[c * 64] = P;
    mine[(C + c) * 64] = H;
  }
  __syncthreads();
  if (wave == 0) {
    const int64_t pitch = a.batch * p.groups * (64 * C), place = (b * p.groups + group) * (64 * C) + lane * C;
    const bool ends_run = SPLIT && seg % kRun == kRun - 1;
    float h[C];
#pragma unroll
    for (int c = 0; c < C; ++c) h[c] = a.h0 ? a.h0[b * a.dim + at + c] : 0.0f;
    if (SPLIT) {
      if (!ends_run) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float P, H;
          join<1>(lds + c * 64 + lane, C * 64, 2 * 64 * C, waves, P, H);
          publish(p.maps + seg * pitch + place + c, map_bits(P), H);
        }
      }
      enter<C>(p.maps + place, p.states + place, pitch, seg, h);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) hand_on<1>(lds + c * 64 + lane, C * 64, 2 * 64 * C, waves, h[c]);
    if (ends_run) {
#pragma unroll
      for (int c = 0; c < C; ++c) publish(p.states + int64_t(seg / kRun) * pitch + place + c, 0, h[c]);
    }
    if (!OUT) {
#pragma unroll
      for (int c = 0; c < C; ++c) p.entry[(seg + 1) * pitch + place + c] = h[c];
    }
    if (OUT && seg == p.nseg - 1 && on) {
#pragma unroll
      for (int c = 0; c < C; ++c) a.h_last[b * a.dim + ch + c] = h[c];
    }
  }
  if (!OUT) return;
  __syncthreads();
  float h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) h[c] = mine[c * 64];
  IO* out = static_cast<IO*>(a.out) + b * a.len * a.dim + ch;
#pragma unroll
  for (int j = 0; j < T; ++j) {
    float y[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      h[c] = fmaf(A[j][c], h[c], U[j][c]);
      y[c] = h[c];
      if (ZGATE) {
        const float q = z[j].get(c);
        y[c] *= q * sigmoid(q);
      }
      if (j >= span.live) y[c] = 0.0f;
    }
    if (on && span.k0 + j < a.len) *reinterpret_cast<V*>(out + span.place(j) * a.dim) = packed<IO, C>(y);
  }
}

}  // namespace rec
}  // namespace sscan
