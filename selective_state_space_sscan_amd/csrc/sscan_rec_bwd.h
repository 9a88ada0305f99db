// sscan_rec_bwd.h -- gradients of the gated recurrence.  Where rows have several segments, a
// first kernel leaves the states that enter them (sscan_rec_fwd.h, without its outputs); the
// kernel below then takes the segments of a row at once, the last ones first, and joins the
// adjoints between them as the forward pass joins the states.  2 x 4096 x 2560 bf16 takes 149 us;
// in a trace, which adds to both, the states take 51 and the gradients 104 (vector units 63%
// busy, 3.6 TB/s).
#pragma once

#include "sscan_rec_fwd.h"

namespace sscan {
namespace rec {

// A segment has 64 tokens: a wave as many as the registers hold without spilling any, a block
// the waves for the others; four channels a lane where the inputs come in 8 bits, for whole
// words of them.  Segments of 32 tokens spend more on the words between them (4 x 4096 x 2048
// from 8 bits 301 us a call, so 265).
constexpr int kBackSegment = 64;
constexpr int back_tokens(bool kept) { return kept ? 4 : 8; }
inline int back_channels(int64_t dim, bool kept, bool io_bf16) {
  return kept && io_bf16 && dim % 4 == 0 ? 4 : channels_of(dim);
}
constexpr int state_tokens(int c, bool kept, bool few) { return few || c == 4 || (c == 2 && kept) ? 8 : 16; }
// Waves of a block in the kernel of the states: gradients of 8 x 4096 x 2048 bf16 with sixteen
// 414 us, with eight 402.
constexpr int kStateWaves = 8;

// One segment a block.  The adjoint that passes from token t to t - 1 is c_t = a_t (e_t +
// c_{t+1}), e_t = dout_t silu(z_t): a map of the adjoint that enters a tile from behind, with
// the same product of decays as the state's.  A lane holds its tokens' inputs as they were
// loaded and 1 - a (a itself where it has no rounding to lose), walks them once for both
// maps, and after the exchange once forwards from the state before them and once back.
template <typename IO, int C, int T, bool GATED, bool IGATE, bool ZGATE, bool KEPT>
__global__ __launch_bounds__(64 * kBackSegment / T) void bwd_kernel(TileArgs p, RecBwdArgs w, float* partial) {
  extern __shared__ float lds[];     // [waves][4][64 C]: A and H of the states, A and H of the adjoints
  __shared__ unsigned number;
  constexpr int kPlane = 64 * C, kPitch = 4 * kPlane;
  const RecArgs& a = p.a;
  const int lane = int(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int waves = int(blockDim.x) >> 6;
  const Tile tile = Tile::of(p, &number, true);
  const int seg = tile.seg;
  const bool split = p.nseg > 1;     // rows have several segments
  const int64_t b = tile.b, group = tile.group;
  const int64_t ch = (group * 64 + lane) * C;
  const bool on = ch < a.dim;
  const int64_t at = on ? ch : 0;
  const Span span(a, b, (int64_t(seg) * waves + wave) * T, T);
  const int64_t pitch = a.batch * p.groups * kPlane, place = (b * p.groups + group) * kPlane + lane * C;

  float rate[C];
#pragma unroll
  for (int c = 0; c < C; ++c) rate[c] = GATED ? decay_rate(a.lam, at + c, a.c) : 0.0f;
  const bool far = any_far<C>(rate);

  In<IO, C, KEPT> x[T], g[T], i[T], z[T];
  In<IO, C, false> d[T];
  // sigmoid(i) in the place of i, where registers are left (8 bits and their scales take more)
  constexpr bool kHold = IGATE && !KEPT, kLate = KEPT;
  float S[kHold ? T : 1][C];
  float D[T][C], U[T][C];            // 1 - a (or a) and the token's input; later the state before the token
  const auto decay_of = [&](float v) { return GATED ? 1.0f - v : v; };
  float P[C], H[C], M[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    P[c] = 1.0f;
    H[c] = M[c] = 0.0f;
  }
  if (span.live > 0) {
    const Rows rows(span);
    const Loader<IO, C, KEPT> gs(a, a.g, a.kept.g, a.kept.gs, b, span, at), xs(a, a.x, a.kept.x, a.kept.xs, b, span, at),
        is(a, a.i, a.kept.i, a.kept.is, b, span, at), zs(a, a.z, a.kept.z, a.kept.zs, b, span, at);
    const RecIn back{w.dout, a.len * a.dim, a.dim};
    const Loader<IO, C, false> ds(a, back, nullptr, nullptr, b, span, at);
    // token by token: the first are computed while the last are on their way
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const unsigned k = rows.at(j);
      g[j] = gs.row(k);
      if (IGATE) i[j] = is.row(k);
      x[j] = xs.row(k);
      __builtin_amdgcn_sched_barrier(0);
    }
    const auto load_back = [&] {
#pragma unroll
      for (int j = T - 1; j >= 0; --j) {
        const unsigned k = rows.at(j);
        d[j] = ds.row(k);
        if (ZGATE) z[j] = zs.row(k);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    if (!kLate) load_back();
#pragma unroll
    for (int j = 0; j < T; ++j) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const Decay q = decay<GATED>(g[j].get(c), rate[c], far);
        float u = x[j].get(c);
        if (GATED) u *= q.w;
        if (IGATE) {
          const float s = sigmoid(i[j].get(c));
          u *= s;
          if (kHold) S[j][c] = s;
        }
        D[j][c] = GATED ? q.loss : q.a;
        U[j][c] = u;
        if (C == 4) __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (kLate) load_back();
    if (span.live < T) {             // tokens past the row's end leave state and adjoint alone
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (j >= span.live) {
            D[j][c] = GATED ? 0.0f : 1.0f;
            U[j][c] = 0.0f;
          }
    }
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float A = decay_of(D[j][c]);
        P[c] *= A;
        H[c] = fmaf(A, H[c], U[j][c]);
      }
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      if (j < span.live) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float e = d[j].get(c);
          if (ZGATE) {
            const float v = z[j].get(c);
            e *= v * sigmoid(v);
          }
          M[c] = decay_of(D[j][c]) * (M[c] + e);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  as_loaded(g);
  as_loaded(x);
  if (IGATE && !kHold) as_loaded(i);
  as_loaded(d);
  if (ZGATE) as_loaded(z);
  float* mine = lds + wave * kPitch + lane;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    mine[c * 64] = mine[2 * kPlane + c * 64] = P[c];
    mine[kPlane + c * 64] = H[c];
    mine[3 * kPlane + c * 64] = M[c];
  }
  __syncthreads();
  if (wave == 0) {                   // adjoints, from the last wave on
    const int back = p.nseg - 1 - seg;
    const bool ends_run = split && back % kRun == kRun - 1;
    float* first = lds + 2 * kPlane + lane;
    float h[C];
    if (back == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) h[c] = w.dh_last ? w.dh_last[b * a.dim + at + c] : 0.0f;
    } else {
      if (!ends_run) {
        float A[C], B[C];
        join<-1, C>(first, kPlane, kPitch, waves, A, B);
#pragma unroll
        for (int c = 0; c < C; ++c) publish(p.maps + back * pitch + place + c, map_bits(A[c]), B[c]);
      }
      enter<C>(p.maps + place, p.states + place, pitch, back, h);
    }
    hand_on<-1, C>(first, kPlane, kPitch, waves, h);
    if (split && (back == 0 || ends_run)) {
      uint64_t* to = ends_run ? p.states + int64_t(back / kRun) * pitch : p.maps;
#pragma unroll
      for (int c = 0; c < C; ++c) publish(to + place + c, 0, h[c]);
    }
    if (w.dh0 && seg == 0 && on) {
#pragma unroll
      for (int c = 0; c < C; ++c) w.dh0[b * a.dim + ch + c] = h[c];
    }
  }
  if (wave == waves - 1) {           // states, from the first wave on
    float h[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      h[c] = seg > 0 ? p.entry[seg * pitch + place + c] : a.h0 ? a.h0[b * a.dim + at + c] : 0.0f;
    hand_on<1, C>(lds + lane, kPlane, kPitch, waves, h);
  }
  __syncthreads();
  float h[C], carry[C], dlam[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    h[c] = mine[c * 64];
    carry[c] = mine[2 * kPlane + c * 64];
    dlam[c] = 0.0f;
  }
  if (span.live > 0) {
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float before = h[c];
        h[c] = fmaf(decay_of(D[j][c]), h[c], U[j][c]);
        U[j][c] = before;
      }
  }
  const int64_t row = b * a.len * a.dim * int64_t(sizeof(IO));
  const unsigned step = unsigned(a.dim) * unsigned(sizeof(IO)), lane_at = unsigned(ch) * unsigned(sizeof(IO));
  const Rows rows(span);
  const int64_t lowest = row + (span.live > 0 ? rows.lowest(span) : 0) * a.dim * int64_t(sizeof(IO));
  const auto put = [&](void* out, int j, const float (&v)[C]) {
    store_any<IO, C>(reinterpret_cast<IO*>(static_cast<char*>(out) + lowest + (rows.at(j) * step + lane_at)),
                     packed<IO, C>(v));
  };
#pragma unroll
  for (int j = T - 1; j >= 0; --j) {
    float ox[C] = {}, og[C] = {}, oi[C] = {}, oz[C] = {};
    if (j < span.live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float A = decay_of(D[j][c]), before = U[j][c];
        const float v = x[j].get(c), s = kHold ? S[kHold ? j : 0][c] : IGATE ? sigmoid(i[j].get(c)) : 1.0f;
        float e = d[j].get(c);
        if (ZGATE) {
          const float q = z[j].get(c), sq = sigmoid(q);
          oz[c] = e * h[c] * sq * fmaf(q, 1.0f - sq, 1.0f);
          e *= q * sq;
        }
        h[c] = before;               // the state after the token before
        const float adj = e + carry[c];
        carry[c] = A * adj;
        float dlog = carry[c] * before, wgt = 1.0f;
        const float sx = s * v;
        if (GATED) {
          const float loss = D[j][c], r = sigmoid(g[j].get(c));
          // 1 / w; the instruction answers infinity for what is no normal number, whose w is taken as 0
          const float w2 = loss * (2.0f - loss), inv = w2 >= 0x1p-126f ? __builtin_amdgcn_rsqf(w2) : 0.0f;
          wgt = w2 * inv;
          dlog = fmaf(-adj * sx, A * A * inv, dlog);
          og[c] = -dlog * rate[c] * r * (1.0f - r);
          dlam[c] = fmaf(-dlog, r, dlam[c]);
        } else {
          og[c] = dlog;
        }
        const float dw = adj * wgt;
        ox[c] = dw * s;
        oi[c] = dw * sx * (1.0f - s);
        if (C == 4) __builtin_amdgcn_sched_barrier(0);  // four channels side by side would spill
      }
    }
    if (on && j < span.live) {
      put(w.dx, j, ox);
      put(w.dg, j, og);
      if (IGATE) put(w.di, j, oi);
      if (ZGATE) put(w.dz, j, oz);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (span.live < T) {               // zeros past the row's end
    for (int j = span.live; j < T; ++j) {
      if (!on || span.k0 + j >= a.len) continue;
      const int64_t to = row + (span.k0 + j) * a.dim * int64_t(sizeof(IO)) + lane_at;
      const auto zero = [&](void* out) {
        store_any<IO, C>(reinterpret_cast<IO*>(static_cast<char*>(out) + to), typename Vec<IO, C>::V{});
      };
      zero(w.dx);
      zero(w.dg);
      if (IGATE) zero(w.di);
      if (ZGATE) zero(w.dz);
    }
  }
  if (GATED && w.dlam) {             // over the block's waves, in order
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) mine[c * 64] = dlam[c];
    __syncthreads();
    if (wave == 0 && on) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float sum = 0.0f;
        for (int v = 0; v < waves; ++v) sum += lds[v * kPitch + c * 64 + lane];
        const float l = a.lam[ch + c];
        partial[(int64_t(seg) * a.batch + b) * a.dim + ch + c] = sum * (a.c / (1.0f + expf(-l)));
      }
    }
  }
}

struct BackPlan {
  int c, waves;
  bool few;
  int64_t groups, nseg;
  int64_t words;                     // words of one set of maps and states
  size_t off_words, off_entry, off_partial, bytes;
};

inline BackPlan back_plan(int64_t batch, int64_t len, int64_t dim, bool kept, bool io_bf16) {
  BackPlan p;
  p.c = back_channels(dim, kept, io_bf16);
  p.groups = up(dim, 64 * p.c);
  p.few = few_tiles(batch, len, p.groups);
  const int64_t row = batch * p.groups * 64 * p.c;
  p.nseg = up(len, kBackSegment);
  p.waves = p.nseg > 1 ? kBackSegment / back_tokens(kept) : int(up(len, back_tokens(kept)));
  p.words = p.nseg > 1 ? (p.nseg + p.nseg / kRun) * row : 0;
  p.off_words = 256;
  p.off_entry = p.off_words + size_t(p.words) * 16;
  p.off_partial = p.off_entry + (p.nseg > 1 ? size_t(p.nseg * row) * 4 : 0);
  p.bytes = (p.off_partial + size_t(p.nseg) * size_t(batch) * size_t(dim) * 4 + 255) / 256 * 256;
  return p;
}

template <typename IO, int C, bool KEPT>
hipError_t bwd(const RecBwdArgs& w, const BackPlan& plan, char* workspace, hipStream_t stream) {
  const RecArgs& a = w.f;
  const int64_t row = a.batch * plan.groups * 64 * C;
  uint64_t* words = reinterpret_cast<uint64_t*>(workspace + plan.off_words);
  unsigned* ticket = reinterpret_cast<unsigned*>(workspace);
  float* partial = reinterpret_cast<float*>(workspace + plan.off_partial);
  TileArgs p{a, words, words + plan.nseg * row, ticket, reinterpret_cast<float*>(workspace + plan.off_entry),
             0, int(plan.nseg), unsigned(plan.groups)};
  const bool split = plan.nseg > 1, igate = KEPT ? a.kept.i != nullptr : a.i.p != nullptr,
             zgate = KEPT ? a.kept.z != nullptr : a.z.p != nullptr;
  if (split) {
    const int64_t n = plan.words, blocks = up(n, 256 * 4);
    clear_kernel<<<dim3(unsigned(blocks < 2048 ? blocks : 2048)), 256, 0, stream>>>(reinterpret_cast<uint4*>(words), n,
                                                                                    ticket);
    // before the last segment only; its maps and states need no more room than the adjoints'
    const int each = state_tokens(C, KEPT, plan.few);
    const int64_t tokens = (plan.nseg - 1) * kBackSegment + 1, tiles = up(tokens, each);
    const int waves = tiles < kStateWaves ? int(tiles) : kStateWaves;
    p.nseg = int(up(tiles, waves));
    p.states = p.maps + p.nseg * row;
    p.entry_step = kBackSegment;
    const dim3 grid(unsigned(p.nseg * a.batch * plan.groups));
    by_flag(a.lam != nullptr, [&](auto gated) {
      by_flag(igate, [&](auto ig) {
        const auto with = [&](auto t) {
          fwd_kernel<IO, C, decltype(t)::value, decltype(gated)::value, decltype(ig)::value, false, false, KEPT, false>
              <<<grid, waves * 64, size_t(waves) * 2 * 64 * C * 4, stream>>>(p);
        };
        if (each == 8)
          with(std::integral_constant<int, 8>());
        else if constexpr (state_tokens(C, KEPT, false) == 16)
          with(std::integral_constant<int, 16>());
      });
    });
    p.maps += plan.words;
    p.states = p.maps + plan.nseg * row;
    p.nseg = int(plan.nseg);
    ++p.ticket;
  }
  const dim3 grid(unsigned(plan.nseg * a.batch * plan.groups));
  by_flag(a.lam != nullptr, [&](auto gated) {
    by_flag(igate, [&](auto ig) {
      by_flag(zgate, [&](auto zg) {
        bwd_kernel<IO, C, back_tokens(KEPT), decltype(gated)::value, decltype(ig)::value, decltype(zg)::value, KEPT>
            <<<grid, plan.waves * 64, size_t(plan.waves) * 4 * 64 * C * 4, stream>>>(p, w, partial);
      });
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !w.dlam) return e;
  float* const out[1] = {w.dlam};
  return launch_row_sums(partial, out, 1, a.dim, plan.nseg * a.batch, stream);
}

// The call whose inputs come in 8 bits (sscan_rec_bwd_kept.hip).
hipError_t launch_bwd_kept(const RecBwdArgs& w, const BackPlan& plan, char* workspace, hipStream_t stream);

}  // namespace rec
}  // namespace sscan
