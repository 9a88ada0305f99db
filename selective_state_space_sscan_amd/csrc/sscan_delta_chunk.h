// sscan_delta_chunk.h -- the gated delta rule's walk over chunks, shared by the forward
// pass and by the recomputation of the states in the backward pass.
#pragma once

#include "sscan_delta.h"
#include "sscan_delta_device.h"

namespace sscan {
namespace delta {

// A chunk's rows of K (or Q) on their way from memory to the LDS tile, by kThreads
// threads, held in registers meanwhile.
template <typename IO, int KP, int kThreads>
struct RowsAhead {
  static constexpr int kUnits = kC * KP / 8 / kThreads;
  typename Io<IO>::V8 x[kUnits];

  __device__ __forceinline__ void load(const IO* p, int64_t stride, int t0, int len, int dk, bool wide) {
    const int live = len - t0 < kC ? len - t0 : kC;
    const Buffer rows = rows_of(p + t0 * stride, live, stride, dk);
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int u = int(threadIdx.x) + kThreads * n, row = u / (KP / 8), unit = u % (KP / 8);
      // rows past the end are told apart by their number: overlapping ones (a token stride
      // below the row's size, 0 for a broadcast) lie inside the buffer
      load8<IO>(rows, (row * int(stride) + 8 * unit) * int(sizeof(IO)), row < live ? dk - 8 * unit : 0, wide, &x[n]);
    }
  }

  // Terms follow each other Tile<KP>::kElems apart.
  __device__ __forceinline__ void store(bf16* tile) const {
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int u = int(threadIdx.x) + kThreads * n;
      bf16* at = tile + Tile<KP>::unit_at(u / (KP / 8), u % (KP / 8));
      const auto f = as_frag(x[n]);
#pragma unroll
      for (int k = 0; k < Io<IO>::kN; ++k) *reinterpret_cast<bf16x8*>(at + k * Tile<KP>::kElems) = f.t[k];
    }
  }
};

// A contiguous block of kBytes, likewise.
template <int kBytes, int kThreads>
struct BytesAhead {
  static constexpr int kUnits = (kBytes / 16 + kThreads - 1) / kThreads;
  u32x4 x[kUnits > 0 ? kUnits : 1];

  __device__ __forceinline__ void load(const char* p) {
    const Buffer b = buffer_of(p, kBytes);
#pragma unroll
    for (int n = 0; n < kUnits; ++n)
      x[n] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int(threadIdx.x) + kThreads * n) * 16, 0, 0));
  }

  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int u = int(threadIdx.x) + kThreads * n;
      if ((n + 1) * kThreads <= kBytes / 16 || u < kBytes / 16) reinterpret_cast<u32x4*>(lds)[u] = x[n];
    }
  }
};

// A wave's sixteen columns of V of a chunk, in the accumulator layout.  bf16: a row of
// them is 32 bytes, lane = token loads them whole, and the wave turns them around in 2 KB
// of LDS of its own (against sixteen 2-byte loads a lane: 0.7 us less a chunk of eight
// waves).  float32: each lane loads its own elements.
template <typename IO>
struct ColumnsAhead {
  static constexpr int kLds = 16;
  IO x[4][4];

  // p: the chunk's first row, of which `live` are read (the others are zeros)
  __device__ __forceinline__ void load(const IO* p, int live, int64_t stride, int col0, int dv, bool) {
    const Buffer rows = rows_of(p, live, stride, dv);
    const int i = lane_id() & 15, first = 8 * (lane_id() >> 4);
    const int at = here(col0 + i < dv ? (first * int(stride) + col0 + i) * int(sizeof(IO)) : kOutside);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 32 * (m >> 1) + 4 * (m & 1) + r;
        load1(rows, first + row < live ? at + row * int(stride) * int(sizeof(IO)) : kOutside, &x[m][r]);
      }
  }

  __device__ __forceinline__ void get(char*, f32x4 (&v)[4]) const {
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[m][r] = to_f32(x[m][r]);
  }
};

template <>
struct ColumnsAhead<bf16> {
  static constexpr int kLds = kC * 16 * 2;  // bytes a wave
  bf16x8 x[2];

  __device__ __forceinline__ void load(const bf16* p, int live, int64_t stride, int col0, int dv, bool wide) {
    const Buffer rows = rows_of(p, live, stride, dv);
#pragma unroll
    for (int n = 0; n < 2; ++n)
      load8<bf16>(rows, (lane_id() * int(stride) + col0 + 8 * n) * 2, lane_id() < live ? dv - col0 - 8 * n : 0, wide, &x[n]);
  }

  __device__ __forceinline__ void get(char* own, f32x4 (&v)[4]) const {
    const int lane = lane_id(), i = lane & 15, qd = lane >> 4;
    bf16* tile = reinterpret_cast<bf16*>(own);
#pragma unroll
    for (int n = 0; n < 2; ++n) *reinterpret_cast<bf16x8*>(tile + 16 * lane + 8 * n) = x[n];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int row = 32 * (m >> 1) + 8 * qd + 4 * (m & 1) + (i >> 2);
      v[m] = __builtin_convertvector(read_tr(tile + 16 * row + 4 * (i & 3)), f32x4);
    }
    __builtin_amdgcn_wave_barrier();
  }
};

// LDS of a walk: per chunk the K tile, the Q tile, the fragments of two triangular
// matrices and the per-token factors.  bf16: two sets, the next chunk's being filled
// while one is read (one barrier a chunk); float32 has room for one (two barriers).
template <typename IO, int KP, bool kWithQ, int kVecs>
struct WalkLds {
  static constexpr int kTileBytes = Io<IO>::kN * Tile<KP>::kElems * 2;
  static constexpr int kBytesT = kFrags * kTerms * kFragBytes, kBytesP = kWithQ ? kBytesT : 0;
  static constexpr int kQ = kTileBytes, kT = kQ + (kWithQ ? kTileBytes : 0), kP = kT + kBytesT, kVec = kP + kBytesP;
  static constexpr int kSet = kVec + kVecs * 4, kSets = std::is_same<IO, bf16>::value ? 2 : 1;
};

// A wave owns sixteen columns of S for the whole sequence (KP x 16, in the accumulator
// layout) and walks the chunks in order; columns are independent, so waves never
// exchange data: every product's result is the next product's B factor in the same
// lane.  A block is W waves (16 W columns) that share the chunk's K and Q tiles and
// the fragments of T and P through LDS; the next chunk's come in while a chunk is
// computed.  V and the output move between memory and the lanes that own them (32-byte
// runs of a row that the block's waves complete to whole lines).
//
// A row is walked in nseg segments at once.  kOut: the output walk, and with the last
// segment the last state; kStates: the backward pass's recomputation, which leaves every
// chunk's entry state [KP][dvp] and U [64][dvp] in float32 instead.  kEnds: the
// segments' transitions S -> M S + N, walked before those two where nseg > 1: the state
// columns from zero (segment 0: from h0) give N, and the columns of the identity without
// values give M.  Blocks nvb .. of a segment hold the identity's columns.
//
// Outputs are computed from float32 factors as the states are, and rounded once: with two
// terms (16 bits) in their products the output walk of 4 x 2048 tokens of 16 heads took 57 us
// and not 62, a document of 32768 650 in all and not 685, and outputs whose parts cancel lost
// up to 2^-16 of the parts.
//
// Bound by the issue of matrix instructions and of the vector ones that cut float32
// factors into terms.  A chunk and 128 columns cost 28.3 MFLOP of products for the output
// walk (17.3 without Q and P), 8.4 as written down.  A document of 32768 tokens of 16 heads
// of 128 x 128: 0.23 TFLOP in 241 to 266 us (0.87 to 0.96 PFLOP/s; a large bf16 product
// reaches 1.18), its transitions, 29 blocks of 32 chunks a head, 0.26 TFLOP in 280 to 312 us
// (0.82 to 0.92).  LDS is not the bound (32 columns a wave, which halves its reads, take as
// long), nor HBM (0.43 GB, 85 us at a large copy's 5.1 TB/s).
enum WalkMode { kOut, kStates, kEnds };

struct WalkArgs {
  int nchunk, nvb, nseg, seg_chunks, dvp, wide;
  const char *frag_t, *frag_p;
  const float* vec;
  float *states, *values;   // kStates
  // N [row, head][nseg][KP][dvp] (as carried: entry states; the last: a copy of h0 where
  // h_last replaces it), M [..][KP][KP]
  float *ends, *moves;
};

template <typename IO, int KP, int W, int MODE>
__global__ __launch_bounds__(64 * W) void delta_chunk_kernel(DeltaArgs a, WalkArgs w, int vecs) {
  constexpr int N = Io<IO>::kN, kThreads = 64 * W, kRing = N == 1 ? 5 : 2;
  constexpr int kTiles = KP / 16, kSteps = KP / 32;
  constexpr bool OUT = MODE == kOut;
  typedef Tile<KP> TileK;
  typedef WalkLds<IO, KP, OUT, kVecFloats> Lds;
  __shared__ __attribute__((aligned(256))) char lds[Lds::kSets * Lds::kSet];
  __shared__ __attribute__((aligned(16))) char lds_v[W * ColumnsAhead<IO>::kLds];

  const int tid = int(threadIdx.x), lane = tid & 63, wave = wave_id(), i = lane & 15, qd = lane >> 4;
  const int blocks = w.nvb + (MODE == kEnds ? (KP + 16 * W - 1) / (16 * W) : 0);
  // blocks of a segment, which read the same keys and factors, are neighbours
  const unsigned blk = xcd_block();
  const int vb = int(blk % unsigned(blocks)), seg = int(blk / unsigned(blocks) % unsigned(w.nseg));
  const int64_t bh = blk / unsigned(blocks) / unsigned(w.nseg), b = bh / a.hv, at_seg = bh * w.nseg + seg;
  const bool ident = MODE == kEnds && vb >= w.nvb;
  // The last state may replace the entry state, which the output walk's blocks of the first
  // segment read while those of the last one write it.  Walked in segments, they read a copy
  // that the transitions' launch leaves in the last segment's place, which has no end state.
  const bool in_place = w.nseg > 1 && a.h0 && a.h0 == a.h_last, copies = MODE == kEnds && seg == w.nseg - 1;
  if (MODE == kEnds && ((copies && (ident || !in_place)) || (ident && seg == 0))) return;  // nobody reads these
  const int h = int(bh % a.hv), hq = h / (a.hv / a.hk);
  const int col = (ident ? vb - w.nvb : vb) * (16 * W) + 16 * wave + i;
  const int L = int(a.len), Lb = row_len(a.lengths, b, a.len);
  const int first = seg * w.seg_chunks, live_chunks = (Lb + kC - 1) / kC;
  // chunks first .. past - 1
  const int past = copies ? first : live_chunks < first + w.seg_chunks ? live_chunks : first + w.seg_chunks;
  const IO* kp = static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h;
  const IO* qp = static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h;
  const IO* vp = static_cast<const IO*>(a.v) + b * a.sv.b + h * a.sv.h;
  IO* op = static_cast<IO*>(a.out) + (b * a.len * a.hv + h) * a.dv;
  const int64_t out_t = int64_t(a.hv) * a.dv;
  const bool wide_qk = w.wide & 1, wide_v = w.wide & 2, live_col = !ident && col < a.dv;
  // byte offset of this lane's first token (8 qd) and column in a chunk's output rows; its
  // other tokens are 32 (m >> 1) + 4 (m & 1) + r rows on
  const int o_lane = live_col ? (8 * qd * int(out_t) + col) * int(sizeof(IO)) : kOutside;
  const int o_row = int(out_t) * int(sizeof(IO));
  // this lane's elements in a tile: rows by contraction step, columns by pairs of tiles
  int at_row[kSteps], at_col[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    at_row[s] = TileK::unit_at(chained(0, i), 4 * s + qd);
    at_col[s] = TileK::unit_at(8 * qd + (i >> 2), 4 * s + (i & 3));
  }

  const int s_lane = live_col ? (8 * qd * a.dv + col) * 4 : kOutside;
  const int w_lane = !ident && col < w.dvp ? (8 * qd * w.dvp + col) * 4 : kOutside;
  const uint32_t state_bytes = uint32_t(a.dk * a.dv * 4);

  f32x4 S[kTiles] = {};
  if (ident) {
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[m][r] = chained(m, 4 * qd + r) == col ? 1.0f : 0.0f;
  } else if (copies || (seg == 0 && !(OUT && in_place))) {
    if (a.h0) load_state(buffer_of(a.h0 + bh * a.dk * a.dv, state_bytes), s_lane, a.dv, S);
  } else if (MODE != kEnds) {
    const int64_t from = seg == 0 ? at_seg + w.nseg - 1 : at_seg - 1;
    load_state(buffer_of(w.ends + from * KP * w.dvp, KP * w.dvp * 4), w_lane, w.dvp, S);
  }

  RowsAhead<IO, KP, kThreads> next_k, next_q;
  BytesAhead<Lds::kBytesT, kThreads> next_t;
  BytesAhead<Lds::kBytesP, kThreads> next_p;
  ColumnsAhead<IO> next_v;
  f32x4 next_vec = {};
  const auto load_rows = [&](int c) {
    const int t0 = c * kC;
    next_k.load(kp, a.sk.t, t0, Lb, a.dk, wide_qk);
    if constexpr (OUT) next_q.load(qp, a.sq.t, t0, Lb, a.dk, wide_qk);
    next_v.load(vp + t0 * a.sv.t, Lb - t0 < kC ? Lb - t0 : kC, a.sv.t, ident ? a.dv : col - i, a.dv, wide_v);
  };
  const auto load_frags = [&](int c) {
    const int64_t idx = bh * w.nchunk + c;
    next_t.load(w.frag_t + idx * Lds::kBytesT);
    if constexpr (OUT) next_p.load(w.frag_p + idx * Lds::kBytesP);
    if (tid < kVecFloats / 4) next_vec = reinterpret_cast<const f32x4*>(w.vec + idx * vecs)[tid];
  };
  const auto store_rows = [&](char* set) {
    next_k.store(reinterpret_cast<bf16*>(set));
    if constexpr (OUT) next_q.store(reinterpret_cast<bf16*>(set + Lds::kQ));
  };
  const auto store_frags = [&](char* set) {
    next_t.store(set + Lds::kT);
    if constexpr (OUT) next_p.store(set + Lds::kP);
    if (tid < kVecFloats / 4) reinterpret_cast<f32x4*>(set + Lds::kVec)[tid] = next_vec;
  };
  if (first < past) {
    load_rows(first);
    load_frags(first);
    if (Lds::kSets == 2) {
      store_rows(lds + (first & 1) * Lds::kSet);
      store_frags(lds + (first & 1) * Lds::kSet);
    }
  }

  for (int c = first; c < past; ++c) {
    const int t0 = c * kC;
    const int64_t idx = bh * w.nchunk + c;
    const char* set = lds + (Lds::kSets == 2 ? (c & 1) * Lds::kSet : 0);
    char* other = lds + (Lds::kSets == 2 ? (~c & 1) * Lds::kSet : 0);
    f32x4 x[4];
    next_v.get(lds_v + wave * ColumnsAhead<IO>::kLds, x);
    __syncthreads();
    if (Lds::kSets == 1) {
      store_rows(lds);
      store_frags(lds);
      __syncthreads();
    }
    const bool more = c + 1 < past;
    if (more) {
      load_rows(c + 1);
      if (Lds::kSets == 1) load_frags(c + 1);
    }
    if constexpr (MODE == kStates)
      store_state(buffer_of(w.states + idx * KP * w.dvp, KP * w.dvp * 4), w_lane, w.dvp, S);
    const bf16 *sk = reinterpret_cast<const bf16*>(set), *sq = reinterpret_cast<const bf16*>(set + Lds::kQ);
    const char *st = set + Lds::kT + lane * 16, *sp = set + Lds::kP + lane * 16;
    const float* svec = reinterpret_cast<const float*>(set + Lds::kVec);

    // fragments of rows of K and Q, in the order of the products
    struct Rows {
      Frag<N> k, q;
    };
    const auto read_rows = [&](int j, Rows& f) {
      const int at = chained(j / kSteps, 0) * KP + at_row[j % kSteps];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        f.k.t[n] = row_frag(sk + n * TileK::kElems + at);
        if constexpr (OUT) f.q.t[n] = row_frag(sq + n * TileK::kElems + at);
      }
    };
    constexpr int kRingT = 4;
    const auto read_t = [&](int j, Frag<3>& f) {
#pragma unroll
      for (int n = 0; n < 3; ++n) f.t[n] = *reinterpret_cast<const bf16x8*>(st + (j * 3 + n) * kFragBytes);
    };
    const auto read_p = [&](int j, Frag<3>& f) {
#pragma unroll
      for (int n = 0; n < 3; ++n) f.t[n] = *reinterpret_cast<const bf16x8*>(sp + (j * 3 + n) * kFragBytes);
    };
    const auto read_cols = [&](int j, Frag<N>& f) {
      const int m = j >> 1, s = j & 1;
#pragma unroll
      for (int n = 0; n < N; ++n)
        f.t[n] = col_frag(sk + n * TileK::kElems + 32 * s * KP + at_col[m >> 1] + 4 * (m & 1), KP);
    };

    // x = v - c (K S), o = e (Q S), per tile of sixteen tokens in chained order
    Rows rows_ring[kRing];
    ring_start<4 * kSteps>(rows_ring, read_rows);
    Frag<3> sf[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) sf[s] = split(S[2 * s], S[2 * s + 1]);
    f32x4 o[4] = {}, ks = {};
    ring_run<4 * kSteps>(rows_ring, read_rows, [&](int j, const Rows& f) {
      const int m = j / kSteps, s = j % kSteps, tok = chained(m, 4 * qd);
      ks = mul(f.k, sf[s], s == 0 ? f32x4{} : ks);
      if constexpr (OUT) o[m] = mul(f.q, sf[s], o[m]);
      if (s == kSteps - 1) {
        x[m] -= *reinterpret_cast<const f32x4*>(&svec[tok]) * ks;
        if constexpr (OUT) o[m] *= *reinterpret_cast<const f32x4*>(&svec[2 * kC + tok]);
      }
    });
    Frag<3> t_ring[kRingT];
    ring_start<kFrags>(t_ring, read_t);
    if (Lds::kSets == 2 && more) {
      store_rows(other);
      load_frags(c + 1);
    }
    // u = (T diag(beta)) x
    const Frag<3> xf[2] = {split(x[0], x[1]), split(x[2], x[3])};
    f32x4 u[4] = {};
    ring_run<kFrags>(t_ring, read_t,
                     [&](int j, const Frag<3>& f) { u[lower_m(j)] = mul(f, xf[lower_s(j)], u[lower_m(j)]); });
    // o += P u
    if constexpr (OUT) {
      Frag<3> p_ring[kRingT];
      ring_start<kFrags>(p_ring, read_p);
      const Frag<3> uf[2] = {split(u[0], u[1]), split(u[2], u[3])};
      ring_run<kFrags>(p_ring, read_p,
                       [&](int j, const Frag<3>& f) { o[lower_m(j)] = mul(f, uf[lower_s(j)], o[lower_m(j)]); });
      // a state that is not finite times the zero queries past the row's end is none of theirs
      if (Lb - t0 < kC)
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[m][r] = chained(m, 4 * qd + r) < Lb - t0 ? o[m][r] : 0.0f;
      const Buffer rows = rows_of(op + t0 * out_t, L - t0 < kC ? L - t0 : kC, out_t, a.dv);
      const int at = here(o_lane);
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) store1(rows, at + (32 * (m >> 1) + 4 * (m & 1) + r) * o_row, IO(o[m][r]));
    } else if constexpr (MODE == kStates) {
      store_state(buffer_of(w.values + idx * kC * w.dvp, kC * w.dvp * 4), w_lane, w.dvp, u);
    }
    // S = last S + K^T (d u)
    Frag<N> c_ring[kRing];
    ring_start<2 * kTiles>(c_ring, read_cols);
#pragma unroll
    for (int m = 0; m < 4; ++m) u[m] *= *reinterpret_cast<const f32x4*>(&svec[kC + chained(m, 4 * qd)]);
    const Frag<3> df[2] = {split(u[0], u[1]), split(u[2], u[3])};
    const float last = svec[3 * kC];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) S[m] *= last;
    ring_run<2 * kTiles>(c_ring, read_cols, [&](int j, const Frag<N>& f) { S[j >> 1] = mul(f, df[j & 1], S[j >> 1]); });
    if (Lds::kSets == 2 && more) store_frags(other);
  }
  if constexpr (MODE == kEnds) {
    if (ident)
      store_state(buffer_of(w.moves + at_seg * KP * KP, KP * KP * 4), col < KP ? (8 * qd * KP + col) * 4 : kOutside, KP, S);
    else
      store_state(buffer_of(w.ends + at_seg * KP * w.dvp, KP * w.dvp * 4), w_lane, w.dvp, S);
  }
  if constexpr (OUT) {
    // tokens past the row's length: zeros (those of its last chunk were written above)
    const int from = (first < live_chunks ? past : first) * kC, to = (first + w.seg_chunks) * kC;
    if (live_col)
      for (int t = from + qd; t < L && t < to; t += 4) op[t * out_t + col] = IO(0.0f);
    if (seg == w.nseg - 1) store_state(buffer_of(a.h_last + bh * a.dk * a.dv, state_bytes), s_lane, a.dv, S);
  }
}

// The chain over segments: X_j += M_j X_(j-1) for j = 1 .. nseg - 2 (REV: X_j += M_j^T
// X_(j+1) downwards), X the state columns left by the segments.  A step waits for the
// one before it, so as little as possible lies on that path: a block has sixteen columns,
// each of its KP / 32 waves computes 32 rows of them, and takes its rows of M straight to
// its lanes, cut into terms before the step that needs them; only the columns' terms
// (3 KB a wave) go round through LDS, one barrier a step.  Bound by that chain: 64 heads of 4
// segments 14 us, 16 heads of 16 segments 50 us (3.5 us a step, of 14).
template <int KP, bool REV>
__global__ __launch_bounds__(2 * KP) void delta_carry_kernel(const float* moves, float* x, int nseg, int dvp) {
  constexpr int kSteps = KP / 32;
  __shared__ __attribute__((aligned(16))) bf16 terms[2][kSteps][3][64 * 8];
  const int lane = lane_id(), wave = wave_id(), i = lane & 15, qd = lane >> 4;
  // the blocks of a head, which all read its M, are neighbours
  const unsigned ncol = unsigned(dvp) / 16, blk = xcd_block(), head = blk / ncol;
  const int64_t bh = head;
  const int col = int(blk - head * ncol) * 16 + i, steps = nseg - 2;
  const int start = REV ? nseg - 2 : 1, step = REV ? -1 : 1;
  const int x_at = ((32 * wave + 8 * qd) * dvp + col) * 4;  // rows 8 qd .. + 7 of this wave's 32
  const auto x_of = [&](int j) { return buffer_of(x + (bh * nseg + j) * KP * dvp, KP * dvp * 4); };
  f32x8 raw[2][kSteps];
  f32x4 S[2], add[2];
  Frag<3> m[2][kSteps];
  const auto load = [&](int j) {
    const Buffer b = buffer_of(moves + (bh * nseg + j) * KP * KP, KP * KP * 4);
    const int l = here(lane);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int row = chained(2 * wave + p, l & 15), k0 = 32 * k + 8 * (l >> 4);
        if constexpr (REV) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float y;
            load1(b, ((k0 + e) * KP + row) * 4, &y);
            raw[p][k][e] = y;
          }
        } else {
          load_wide(b, (row * KP + k0) * 4, &raw[p][k]);
        }
      }
    load_state(x_of(j), x_at, dvp, add);
  };
  const auto cut = [&] {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int k = 0; k < kSteps; ++k) m[p][k] = split(raw[p][k]);
  };
  load_state(x_of(start - step), x_at, dvp, S);
  load(start);
  cut();
  for (int n = 0; n < steps; ++n) {
    const int j = start + n * step;
    const Frag<3> own = split(S[0], S[1]);
#pragma unroll
    for (int t = 0; t < 3; ++t) *reinterpret_cast<bf16x8*>(&terms[n & 1][wave][t][8 * lane]) = own.t[t];
    S[0] = add[0];
    S[1] = add[1];
    if (n + 1 < steps) load(j + step);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      Frag<3> f;
#pragma unroll
      for (int t = 0; t < 3; ++t) f.t[t] = row_frag(&terms[n & 1][k][t][8 * lane]);
#pragma unroll
      for (int p = 0; p < 2; ++p) S[p] = mul(m[p][k], f, S[p]);
    }
    store_state(x_of(j), x_at, dvp, S);
    if (n + 1 < steps) cut();
  }
}

}  // namespace delta
}  // namespace sscan
