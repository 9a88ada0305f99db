// sscan_rec_fwd.h -- the recurrence over a segment of a row: the forward's kernel, and that of
// the states between segments, which the backward pass starts from.  Long rows are bound by HBM
// (262144 x 1536 bf16 795 us, 5.1 TB/s; a large copy 5.1), a few rounds of blocks by loads and
// arithmetic that take turns (4 x 2048 x 2560 59 us, 3.5 TB/s).
#pragma once

#include "sscan_pack8.h"
#include "sscan_rec_tile.h"

namespace sscan {
namespace rec {

// The largest of a block of 64 channels, C a lane, in all its lanes: sixteen lanes by DPP,
// rows of sixteen by exchanges.
template <int C>
__device__ __forceinline__ unsigned block_max(unsigned m) {
  m = max(m, unsigned(__builtin_amdgcn_update_dpp(0, int(m), 0xb1, 0xf, 0xf, true)));   // quad_perm 1 0 3 2
  m = max(m, unsigned(__builtin_amdgcn_update_dpp(0, int(m), 0x4e, 0xf, 0xf, true)));   // quad_perm 2 3 0 1
  m = max(m, unsigned(__builtin_amdgcn_update_dpp(0, int(m), 0x141, 0xf, 0xf, true)));  // row_half_mirror
  m = max(m, unsigned(__builtin_amdgcn_update_dpp(0, int(m), 0x140, 0xf, 0xf, true)));  // row_mirror
#pragma unroll
  for (int s = 16; s < 64 / C; s *= 2) m = max(m, unsigned(__shfl_xor(int(m), s)));
  return m;
}

// One segment a block (sscan_rec_tile.h).  A lane first turns its tokens into decays and
// inputs, which it holds in registers with their map; the waves' maps meet in LDS, wave 0
// finds the state that enters the segment (from the row's segments before, where there are
// any) and from it those that enter the waves, and every wave walks its tokens once more,
// now from its state, and answers.  OUT: outputs are wanted, not the states before every
// entry_step-th token alone.  KEPT: the inputs come in 8 bits.  KEEP: they are left in 8 bits.
template <typename IO, int C, int T, bool GATED, bool IGATE, bool ZGATE, bool OUT, bool KEPT, bool KEEP>
__global__ __launch_bounds__(kMaxWaves * 64) void fwd_kernel(TileArgs p) {
  extern __shared__ float lds[];     // [waves][2][64 C]: A and H; then the waves' entry states in A's place
  __shared__ unsigned number;
  const RecArgs& a = p.a;
  const int lane = int(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int waves = int(blockDim.x) >> 6;
  const Tile tile = Tile::of(p, &number);
  const int seg = tile.seg;
  const bool split = p.nseg > 1;     // rows have several segments
  const int64_t b = tile.b, group = tile.group;
  const int64_t ch = (group * 64 + lane) * C;
  const bool on = ch < a.dim;
  const int64_t at = on ? ch : 0;    // lanes beyond the last channel read the first ones
  const Span span(a, b, (int64_t(seg) * waves + wave) * T, T);

  float rate[C];
#pragma unroll
  for (int c = 0; c < C; ++c) rate[c] = GATED ? decay_rate(a.lam, at + c, a.c) : 0.0f;
  const bool far = any_far<C>(rate);

  // A tensor's tokens in 8 bits.  A block of 64 channels lies in kBlockLanes lanes, which all
  // have its largest element; lane j of them takes token j's, so that one evaluation gives all
  // the tile's scales, and hands them back.
  const auto keep = [&](const In<IO, C, KEPT>(&v)[T], int8_t* q, float* s) {
    constexpr int kBlockLanes = 64 / C;
    const int first = lane / kBlockLanes * kBlockLanes, nth = lane - first;
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < T; ++j) {
      unsigned m = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) m = max(m, magnitude(v[j].get(c)));
      m = block_max<C>(on ? m : 0);
      top = nth == j ? m : top;
    }
    const Scale scale(top);
    const int64_t blocks = (a.dim + kPackBlock - 1) / kPackBlock, block = group * C + lane / kBlockLanes;
    if (nth < span.live && block < blocks) s[(b * a.len + span.place(nth)) * blocks + block] = scale.step;
    const Rows rows(span);
    int8_t* to = q + (b * a.len + rows.lowest(span)) * a.dim;  // the same in all lanes
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const float per = __shfl(scale.per, first + j);
      typename Vec<int8_t, C>::V k;
      if constexpr (C == 1) {
        k = steps_of<IO>(v[j].get(0), per);
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c) k[c] = steps_of<IO>(v[j].get(c), per);
      }
      if (j < span.live && on) store_any<int8_t, C>(to + (rows.at(j) * unsigned(a.dim) + unsigned(ch)), k);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  float A[T][C], U[T][C];
  In<IO, C, KEPT> z[T];
  if (span.live > 0) {
    In<IO, C, KEPT> x[T], g[T], i[T];
    const Rows rows(span);
    const Loader<IO, C, KEPT> gs(a, a.g, a.kept.g, a.kept.gs, b, span, at), xs(a, a.x, a.kept.x, a.kept.xs, b, span, at),
        is(a, a.i, a.kept.i, a.kept.is, b, span, at);
    // token by token: the first are computed while the last are on their way
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const unsigned k = rows.at(j);
      g[j] = gs.row(k);
      if (IGATE) i[j] = is.row(k);
      x[j] = xs.row(k);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (KEEP) {
      keep(g, a.kept.g, a.kept.gs);
      keep(x, a.kept.x, a.kept.xs);
      if (IGATE) keep(i, a.kept.i, a.kept.is);
      as_loaded(g);
      as_loaded(x);
      if (IGATE) as_loaded(i);
    }
#pragma unroll
    for (int j = 0; j < T; ++j) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const Decay d = decay<GATED>(g[j].get(c), rate[c], far);
        float u = x[j].get(c);
        if (GATED) u *= d.w;
        if (IGATE) u *= sigmoid(i[j].get(c));
        A[j][c] = d.a;
        U[j][c] = u;
      }
      __builtin_amdgcn_sched_barrier(0);  // a token at a time: several would need more registers than there are
    }
    // on their way while the state comes; with the others they would not fit the registers
    if (OUT && ZGATE) {
      const Loader<IO, C, KEPT> zs(a, a.z, a.kept.z, a.kept.zs, b, span, at);
#pragma unroll
      for (int j = 0; j < T; ++j) {
        z[j] = zs.row(rows.at(j));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (KEEP && ZGATE) {
      keep(z, a.kept.z, a.kept.zs);
      as_loaded(z);
    }
  }
  if (span.live < T) {               // tokens past the row's end leave the state alone
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (j >= span.live) {
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
    const bool ends_run = split && seg % kRun == kRun - 1;
    float h[C];
    if (seg == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) h[c] = a.h0 ? a.h0[b * a.dim + at + c] : 0.0f;
    } else {
      if (!ends_run) {
        float P[C], H[C];
        join<1, C>(lds + lane, C * 64, 2 * 64 * C, waves, P, H);
#pragma unroll
        for (int c = 0; c < C; ++c) publish(p.maps + seg * pitch + place + c, map_bits(P[c]), H[c]);
      }
      enter<C>(p.maps + place, p.states + place, pitch, seg, h);
    }
    hand_on<1, C>(lds + lane, C * 64, 2 * 64 * C, waves, h);
    if (split && (seg == 0 || ends_run)) {
      uint64_t* to = ends_run ? p.states + int64_t(seg / kRun) * pitch : p.maps;
#pragma unroll
      for (int c = 0; c < C; ++c) publish(to + place + c, 0, h[c]);
    }
    if (OUT && seg == p.nseg - 1 && on) {
#pragma unroll
      for (int c = 0; c < C; ++c) a.h_last[b * a.dim + ch + c] = h[c];
    }
  }
  __syncthreads();
  float h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) h[c] = mine[c * 64];
  if (!OUT) {
    if (span.k0 % p.entry_step == 0 && span.k0 < a.len) {
      const int64_t pitch = a.batch * p.groups * (64 * C), place = (b * p.groups + group) * (64 * C) + lane * C;
#pragma unroll
      for (int c = 0; c < C; ++c) p.entry[span.k0 / p.entry_step * pitch + place + c] = h[c];
    }
    return;
  }
  char* row = static_cast<char*>(a.out) + b * a.len * a.dim * int64_t(sizeof(IO));  // the same in all lanes
  const unsigned place = unsigned(ch) * unsigned(sizeof(IO));
  const auto answer = [&](int j) {
    float y[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      h[c] = fmaf(A[j][c], h[c], U[j][c]);
      y[c] = h[c];
      if (ZGATE) {
        const float q = z[j].get(c);
        y[c] *= q * sigmoid(q);
      }
    }
    return packed<IO, C>(y);
  };
  if (span.live > 0) {
    const Rows rows(span);
    char* to = row + rows.lowest(span) * a.dim * int64_t(sizeof(IO));
    const unsigned step = unsigned(a.dim) * unsigned(sizeof(IO));
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const auto y = answer(j);
      if (on && j < span.live) store_any<IO, C>(reinterpret_cast<IO*>(to + (rows.at(j) * step + place)), y);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (span.live < T) {               // zeros past the row's end
    for (int j = span.live; j < T; ++j)
      if (on && span.k0 + j < a.len)
        store_any<IO, C>(reinterpret_cast<IO*>(row + (span.k0 + j) * a.dim * int64_t(sizeof(IO)) + place),
                         typename Vec<IO, C>::V{});
  }
}

constexpr int kWaves = 8;            // of a block where rows have several segments

// Channels a lane, and tokens of a wave's tile: sixteen, which the registers hold without
// spilling any (the tokens' decays and inputs alone are 2 C T); eight of two float32 channels,
// and where a call has too few tiles to fill the chip, so that each takes half as long (calls
// from a graph: 3 x 77 x 384 bf16 7.4 us, with sixteen 8.9; 1 x 200 x 2048 10.1, 14.0; 4 x 1000 x
// 384 13.1, 14.6; 1 x 2048 x 1024 15.5, 15.5).  Rows that are long as well lose: twice the segments
// make twice the links between runs (1 x 16384 of 64 channels 46 us, with sixteen 30).  The same
// whether inputs are kept or not: states are joined at the tiles' ends, and outputs are the same bits.
inline int channels_of(int64_t dim) { return dim % 2 == 0 ? 2 : 1; }
constexpr int64_t kFewTiles = 2048;  // half of what the chip holds at once

inline bool few_tiles(int64_t batch, int64_t len, int64_t groups) { return batch * groups * up(len, 16) < kFewTiles; }
inline int tokens_of(int c, bool io_bf16, bool few) { return few || (c == 2 && !io_bf16) ? 8 : 16; }

struct Plan {
  int c, tokens, waves;
  int64_t groups, nseg, words;       // bytes of the maps and states
};

inline Plan plan_of(int64_t batch, int64_t len, int64_t dim, bool io_bf16) {
  Plan p;
  p.c = channels_of(dim);
  p.groups = up(dim, 64 * p.c);
  p.tokens = tokens_of(p.c, io_bf16, few_tiles(batch, len, p.groups));
  const int64_t tiles = up(len, p.tokens);
  p.waves = tiles <= kMaxWaves ? int(tiles) : kWaves;
  p.nseg = tiles <= kMaxWaves ? 1 : up(tiles, p.waves);
  p.words = p.nseg > 1 ? (p.nseg + p.nseg / kRun) * batch * p.groups * 64 * p.c * 8 : 0;
  return p;
}

template <typename IO, int C, bool KEEP>
hipError_t fwd(const RecArgs& a, const Plan& plan, char* workspace, hipStream_t stream) {
  uint64_t* words = reinterpret_cast<uint64_t*>(workspace + 256);
  const TileArgs p{a, words, words + plan.nseg * a.batch * plan.groups * 64 * C, reinterpret_cast<unsigned*>(workspace),
                   nullptr, 0, int(plan.nseg), unsigned(plan.groups)};
  const dim3 grid(unsigned(plan.nseg * a.batch * plan.groups)), block(unsigned(plan.waves * 64));
  const size_t lds = size_t(plan.waves) * 2 * 64 * C * 4;
  if (plan.nseg > 1) {
    const int64_t n = plan.words / 16, blocks = up(n, 256 * 4);
    clear_kernel<<<dim3(unsigned(blocks < 2048 ? blocks : 2048)), 256, 0, stream>>>(reinterpret_cast<uint4*>(words), n, p.ticket);
  }
  by_flag(a.lam != nullptr, [&](auto gated) {
    by_flag(a.i.p != nullptr, [&](auto igate) {
      by_flag(a.z.p != nullptr, [&](auto zgate) {
        const auto with = [&](auto tokens) {
          fwd_kernel<IO, C, decltype(tokens)::value, decltype(gated)::value, decltype(igate)::value,
                     decltype(zgate)::value, true, false, KEEP><<<grid, block, lds, stream>>>(p);
        };
        if constexpr (C == 2 && sizeof(IO) == 4) {
          with(std::integral_constant<int, 8>());
        } else {
          if (plan.tokens == 8)
            with(std::integral_constant<int, 8>());
          else
            with(std::integral_constant<int, 16>());
        }
      });
    });
  });
  return hipGetLastError();
}

// f(element, channels a lane), as types.
template <typename F>
hipError_t by_lane(int c, bool io_bf16, F f) {
  const auto with = [&](auto io) {
    return c == 2 ? f(io, std::integral_constant<int, 2>()) : f(io, std::integral_constant<int, 1>());
  };
  return io_bf16 ? with(bf16{}) : with(0.0f);
}

// The forward call whose inputs are left in 8 bits (sscan_rec_keep.hip).
hipError_t launch_keep(const RecArgs& a, const Plan& plan, char* workspace, hipStream_t stream);

}  // namespace rec
}  // namespace sscan
