// sscan_delta_bwd.hip -- gradients of the gated delta rule.
//
// Per chunk (symbols of sscan_delta.h; dX the gradient of X, E = dS1 the adjoint of the
// state leaving the chunk, B_ij = D_ij (k_i . k_j) so that A = diag(beta) B):
//   dU   = P^T dO + diag(exp(G_C - G)) K E
//   X~   = T^T dU                       (gradient of diag(beta) (V - exp(G) K S0))
//   dV   = diag(beta) X~
//   dS0  = exp(G_C) E + scale Q^T diag(exp G) dO - K^T diag(beta exp G) X~
//   dQ   = scale (diag(exp G) dO S0^T + (dO U^T . D) K)
//   R    = -(diag(exp G) X~ S0^T + (X~ U^T . D, strictly lower) K)    K read, over beta
//   W    = scale (dO U^T . D)^T Q - (X~ U^T . D)^T diag(beta) K + diag(exp(G_C - G)) U E^T
//   dK   = diag(beta) R + W
//   dbeta_i = X~_i . v_i + k_i . R_i
//   dG_i = q_i . dQ_i + beta_i k_i . R_i - k_i . W_i,  and G_C also gets <E, S1>;
//   dg_t = the sum of dG_i over the chunk's i >= t
// Kernels: the chunk-local factors, the forward walk (entry states and U of every
// chunk), the walk back (E and X~ of every chunk), and per chunk the gradients.  States
// and adjoints are kept for every chunk in float32.
#include "sscan_delta.h"

#include "sscan_delta_chunk.h"
#include "sscan_delta_device.h"
#include "sscan_delta_prep.h"

namespace sscan {
namespace delta {

// ---- the walk back over chunks ------------------------------------------------------
//
// As the forward walk: a wave owns sixteen columns of the adjoint state, and segments
// are walked at once.  ENDS: only the adjoint that a segment hands to the one before it,
// started from zero (the last segment: from dh_last); the transitions between them are
// the forward walk's, transposed.  Bound by the matrix instructions as it is: 2 x 4096
// tokens of 16 heads of 128 x 128 84 us, its ENDS 70 us.
struct WalkBackArgs {
  int nchunk, nvb, nseg, seg_chunks, dvp, wide;
  const char *frag_tt, *frag_pt;
  const float* vec;
  float *adjoints, *xgrad, *back;
};

template <typename IO, int KP, int W, bool ENDS>
__global__ __launch_bounds__(64 * W) void delta_chunk_bwd_kernel(DeltaBwdArgs b_, WalkBackArgs w) {
  constexpr int N = Io<IO>::kN, kTiles = KP / 16, kSteps = KP / 32, kThreads = 64 * W, kVecs = 5 * kC;
  typedef Tile<KP> TileK;
  typedef WalkLds<IO, KP, true, kVecs> Lds;
  __shared__ __attribute__((aligned(256))) char lds[Lds::kSets * Lds::kSet];

  const DeltaArgs& a = b_.f;
  const int tid = int(threadIdx.x), lane = tid & 63, wave = wave_id(), i = lane & 15, qd = lane >> 4;
  const unsigned blk = xcd_block();
  const int vb = int(blk % unsigned(w.nvb)), seg = int(blk / unsigned(w.nvb) % unsigned(w.nseg));
  const int64_t bh = blk / unsigned(w.nvb) / unsigned(w.nseg), b = bh / a.hv, at_seg = bh * w.nseg + seg;
  if (ENDS && seg == 0) return;  // nobody reads it
  const int h = int(bh % a.hv), hq = h / (a.hv / a.hk);
  const int col = vb * (16 * W) + 16 * wave + i, dvp = w.dvp;
  const int Lb = row_len(a.lengths, b, a.len), live_chunks = (Lb + kC - 1) / kC;
  const int first = seg * w.seg_chunks;
  const int past = live_chunks < first + w.seg_chunks ? live_chunks : first + w.seg_chunks;  // chunks past - 1 .. first
  const IO* kp = static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h;
  const IO* qp = static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h;
  const IO* dp = static_cast<const IO*>(b_.dout) + (b * a.len * a.hv + h) * a.dv;
  const int64_t out_t = int64_t(a.hv) * a.dv;
  const bool wide_qk = w.wide & 1, live_col = col < a.dv;
  const int d_lane = live_col ? (8 * qd * int(out_t) + col) * int(sizeof(IO)) : kOutside;
  const int d_row = int(out_t) * int(sizeof(IO));
  int at_row[kSteps], at_col[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    at_row[s] = TileK::unit_at(chained(0, i), 4 * s + qd);
    at_col[s] = TileK::unit_at(8 * qd + (i >> 2), 4 * s + (i & 3));
  }

  const int s_lane = live_col ? (8 * qd * a.dv + col) * 4 : kOutside;
  const int w_lane = col < dvp ? (8 * qd * dvp + col) * 4 : kOutside;
  const uint32_t state_bytes = uint32_t(a.dk * a.dv * 4);

  f32x4 E[kTiles] = {};
  if (seg == w.nseg - 1) {
    if (b_.dh_last) load_state(buffer_of(b_.dh_last + bh * a.dk * a.dv, state_bytes), s_lane, a.dv, E);
  } else if (!ENDS) {
    load_state(buffer_of(w.back + (at_seg + 1) * KP * dvp, KP * dvp * 4), w_lane, dvp, E);
  }

  RowsAhead<IO, KP, kThreads> next_k, next_q;
  BytesAhead<Lds::kBytesT, kThreads> next_t, next_p;
  typename Io<IO>::V8 next_d[2];  // dO of this lane's column, tokens 32 s + 8 qd ..
  f32x4 next_vec = {};
  const auto load_rows = [&](int c) {
    const int t0 = c * kC;
    next_k.load(kp, a.sk.t, t0, Lb, a.dk, wide_qk);
    next_q.load(qp, a.sq.t, t0, Lb, a.dk, wide_qk);
    const Buffer rows = rows_of(dp + t0 * out_t, Lb - t0 < kC ? Lb - t0 : kC, out_t, a.dv);
    const int at = here(d_lane);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        IO x;
        load1(rows, at + (32 * s + j) * d_row, &x);
        next_d[s][j] = x;
      }
  };
  const auto load_frags = [&](int c) {
    const int64_t idx = bh * w.nchunk + c;
    next_p.load(w.frag_pt + idx * Lds::kBytesT);
    next_t.load(w.frag_tt + idx * Lds::kBytesT);
    if (tid < kVecs / 4) next_vec = reinterpret_cast<const f32x4*>(w.vec + idx * kVecFloatsBwd)[tid];
  };
  const auto store_rows = [&](char* set) {
    next_k.store(reinterpret_cast<bf16*>(set));
    next_q.store(reinterpret_cast<bf16*>(set + Lds::kQ));
  };
  const auto store_frags = [&](char* set) {
    next_p.store(set + Lds::kP);
    next_t.store(set + Lds::kT);
    if (tid < kVecs / 4) reinterpret_cast<f32x4*>(set + Lds::kVec)[tid] = next_vec;
  };
  if (first < past) {
    load_rows(past - 1);
    load_frags(past - 1);
    if (Lds::kSets == 2) {
      store_rows(lds + ((past - 1) & 1) * Lds::kSet);
      store_frags(lds + ((past - 1) & 1) * Lds::kSet);
    }
  }

  for (int c = past - 1; c >= first; --c) {
    const int64_t idx = bh * w.nchunk + c;
    const char* set = lds + (Lds::kSets == 2 ? (c & 1) * Lds::kSet : 0);
    char* other = lds + (Lds::kSets == 2 ? (~c & 1) * Lds::kSet : 0);
    const Frag<N> df[2] = {as_frag(next_d[0]), as_frag(next_d[1])};
    f32x8 dof[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) dof[s][j] = to_f32(next_d[s][j]);
    __syncthreads();
    if (Lds::kSets == 1) {
      store_rows(lds);
      store_frags(lds);
      __syncthreads();
    }
    if (c > first) {
      load_rows(c - 1);
      if (Lds::kSets == 1) load_frags(c - 1);
    }
    if constexpr (!ENDS) store_state(buffer_of(w.adjoints + idx * KP * dvp, KP * dvp * 4), w_lane, dvp, E);
    const bf16 *sk = reinterpret_cast<const bf16*>(set), *sq = reinterpret_cast<const bf16*>(set + Lds::kQ);
    const char *st = set + Lds::kT + lane * 16, *sp = set + Lds::kP + lane * 16;
    const float* svec = reinterpret_cast<const float*>(set + Lds::kVec);

    // du = P^T do + d (K E)
    Frag<3> ef[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) ef[s] = split(E[2 * s], E[2 * s + 1]);
    f32x4 x[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      f32x4 ke = {};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        Frag<N> fk;
#pragma unroll
        for (int n = 0; n < N; ++n) fk.t[n] = row_frag(sk + n * TileK::kElems + chained(m, 0) * KP + at_row[s]);
        ke = mul(fk, ef[s], ke);
      }
      x[m] = ke * *reinterpret_cast<const f32x4*>(&svec[kC + chained(m, 4 * qd)]);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (upper_frag(m, s) < 0) continue;
        Frag<3> f;
#pragma unroll
        for (int n = 0; n < 3; ++n)
          f.t[n] = *reinterpret_cast<const bf16x8*>(sp + (upper_frag(m, s) * 3 + n) * kFragBytes);
        x[m] = mul(f, df[s], x[m]);
      }
    }
    if (Lds::kSets == 2 && c > first) {
      store_rows(other);
      load_frags(c - 1);
    }
    // x~ = T^T du
    const Frag<3> xf[2] = {split(x[0], x[1]), split(x[2], x[3])};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      x[m] = f32x4{};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (upper_frag(m, s) < 0) continue;
        Frag<3> f;
#pragma unroll
        for (int n = 0; n < 3; ++n)
          f.t[n] = *reinterpret_cast<const bf16x8*>(st + (upper_frag(m, s) * 3 + n) * kFragBytes);
        x[m] = mul(f, xf[s], x[m]);
      }
    }
    if constexpr (!ENDS) store_state(buffer_of(w.xgrad + idx * kC * dvp, kC * dvp * 4), w_lane, dvp, x);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int tok = chained(m, 4 * qd);
      x[m] *= *reinterpret_cast<const f32x4*>(&svec[tok]) * *reinterpret_cast<const f32x4*>(&svec[4 * kC + tok]) * -1.0f;
    }
    // E = last E + Q^T (e do) - K^T (c beta x~)
    const Frag<3> yf[2] = {split(x[0], x[1]), split(x[2], x[3])};
    Frag<3> gf[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      gf[s] = split(dof[s] * *reinterpret_cast<const f32x8*>(&svec[2 * kC + 32 * s + 8 * qd]));
    const float last = svec[3 * kC];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      E[m] *= last;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int at = 32 * s * KP + at_col[m >> 1] + 4 * (m & 1);
        Frag<N> fk, fq;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          fk.t[n] = col_frag(sk + n * TileK::kElems + at, KP);
          fq.t[n] = col_frag(sq + n * TileK::kElems + at, KP);
        }
        E[m] = mul(fk, yf[s], E[m]);
        E[m] = mul(fq, gf[s], E[m]);
      }
    }
    if (Lds::kSets == 2 && c > first) store_frags(other);
  }
  if constexpr (ENDS) store_state(buffer_of(w.back + at_seg * KP * dvp, KP * dvp * 4), w_lane, dvp, E);
  if (!ENDS && seg == 0 && b_.dh0)
    store_state(buffer_of(b_.dh0 + bh * a.dk * a.dv, state_bytes), s_lane, a.dv, E);
}

// ---- the gradients of a chunk --------------------------------------------------------

template <int kCtrl>
__device__ __forceinline__ float dpp_f32(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kCtrl, 0xf, 0xf, true));
}

// Sums over the sixteen lanes of a row of n values (8 or 16): lane i receives the sum of
// value i (mod n).  Each step exchanges half of what a lane still holds with the lane
// across bit 3, 2, 1, 0 (by the DPP controls that flip it: rotation by 8, half mirror,
// quad permutations), 45 instructions for sixteen sums.
template <int n>
__device__ __forceinline__ float lane_sums(float (&v)[n]) {
  const int i = lane_id();
  if constexpr (n == 16) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = (i & 8 ? v[k + 8] : v[k]) + dpp_f32<0x128>(i & 8 ? v[k] : v[k + 8]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += dpp_f32<0x128>(v[k]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = (i & 4 ? v[k + 4] : v[k]) + dpp_f32<0x141>(i & 4 ? v[k] : v[k + 4]);
#pragma unroll
  for (int k = 0; k < 2; ++k) v[k] = (i & 2 ? v[k + 2] : v[k]) + dpp_f32<0x4e>(i & 2 ? v[k] : v[k + 2]);
  return (i & 1 ? v[1] : v[0]) + dpp_f32<0xb1>(i & 1 ? v[0] : v[1]);
}

// LDS tile of 64 tokens by VS value columns, in units of eight permuted by the row so
// that sixteen consecutive rows read at one unit touch every bank once.
template <int VS>
struct Slab {
  static constexpr int kUnits = VS / 8, kRows = 16 / kUnits, kElems = kC * VS;
  __device__ static __forceinline__ int at(int row, int unit) {
    return row * VS + ((unit ^ (row / kRows % kUnits)) << 3);
  }
};

template <typename IO, int KP, int VS>
struct GradLds {
  static constexpr int N = Io<IO>::kN, kLdG = 72, kG = kC * kLdG;  // a term of a 64 x 64 factor
  // bf16: the three factors dO U^T, X~ U^T and beta X~ U^T side by side; float32: in turn
  static constexpr int kFactors = N == 1 ? 3 : 1;
  static constexpr int kSlabs = (N + 6) * Slab<VS>::kElems;        // dO, U, X~
  static constexpr int kShared = kSlabs > kFactors * 3 * kG ? kSlabs : kFactors * 3 * kG;
};

// One block of eight waves per (batch row, key head, chunk); the value heads that share
// the key head are walked in order and their dq, dk summed in registers.  A wave owns one
// tile of sixteen key dimensions for all tokens (KP = 64: for half of them).  The value
// axis comes in slabs of VS columns: U, X~ (cut into terms once) and dO through LDS, the
// rows of S0 and E that a wave needs straight to its lanes.  2 x 4096 tokens of 16 heads
// (8 key heads) of 128 x 128, 2048 chunks and heads: 252 us, where the bytes (0.32 GB
// counted) take 62 us at a large copy's 5.1 TB/s and the products, 0.096 TFLOP with the
// float32 factors' terms, 81 us (matrix units busy 17% of the cycles): a block's slabs pass
// through LDS in phases that nothing else fills.  A CU holds one block, by its registers (256
// a thread, about 108 of them sums) and its LDS (124 KB; float32 143 KB, which leaves eight
// registers to scratch).
template <typename IO, int KP, int VS>
__global__ __launch_bounds__(512) void delta_grad_kernel(DeltaBwdArgs b_, int nchunk, const float* vec,
                                                         const float* states, const float* adjoints,
                                                         const float* values, const float* xgrad, int dvp, int wide) {
  typedef GradLds<IO, KP, VS> Lds;
  typedef Tile<KP> TileK;
  typedef Slab<VS> SlabV;
  typedef typename Io<IO>::V8 V8;
  constexpr int N = Lds::N, kLdG = Lds::kLdG, kG = Lds::kG, kTilesK = KP / 16, MT = kTilesK / 2;
  __shared__ __attribute__((aligned(256))) bf16 sk[N * TileK::kElems];
  __shared__ __attribute__((aligned(256))) bf16 sq[N * TileK::kElems];
  __shared__ __attribute__((aligned(256))) bf16 shared[Lds::kShared];
  __shared__ __attribute__((aligned(16))) float svec[kVecFloatsBwd];
  __shared__ double gsum[kC];
  __shared__ float sdot[8][4][kC], sxv[kC], sse[8];
  bf16 *sd = shared, *su = shared + N * SlabV::kElems, *sx = su + 3 * SlabV::kElems;

  const DeltaArgs& a = b_.f;
  const int tid = int(threadIdx.x), lane = tid & 63, wave = wave_id(), i = lane & 15, qd = lane >> 4;
  const int kt = wave % kTilesK, m0 = wave / kTilesK * MT;  // key tile, first token tile
  const int c = int(blockIdx.x % unsigned(nchunk));
  const int64_t bhk = blockIdx.x / unsigned(nchunk), b = bhk / a.hk;
  const int hq = int(bhk % a.hk), share = a.hv / a.hk;
  const int L = int(a.len), Lb = row_len(a.lengths, b, a.len), t0 = c * kC;
  const int64_t qk_t = int64_t(a.hk) * a.dk, v_t = int64_t(a.hv) * a.dv;
  const bool wide_qk = wide & 1, wide_v = wide & 2, wide_d = wide & 4, wide_gv = wide & 16;
  const int out_rows = L - t0 < kC ? L - t0 : kC, rows = Lb - t0 < kC ? Lb - t0 : kC;
  IO* dq_out = static_cast<IO*>(b_.dq) + (b * a.len * a.hk + hq) * a.dk;
  IO* dk_out = static_cast<IO*>(b_.dk) + (b * a.len * a.hk + hq) * a.dk;

  if (t0 >= Lb) {  // past the row's length: zeros
    for (int u = tid; u < out_rows * a.dk; u += 512) {
      const int64_t at = (t0 + u / a.dk) * qk_t + u % a.dk;
      dq_out[at] = IO(0.0f);
      dk_out[at] = IO(0.0f);
    }
    for (int hh = 0; hh < share; ++hh) {
      const int64_t h = hq * share + hh;
      IO* dv_out = static_cast<IO*>(b_.dv) + (b * a.len * a.hv + h) * a.dv;
      for (int u = tid; u < out_rows * a.dv; u += 512) dv_out[(t0 + u / a.dv) * v_t + u % a.dv] = IO(0.0f);
      if (tid < out_rows) {
        b_.dg[(b * a.len + t0 + tid) * a.hv + h] = 0.0f;
        b_.dbeta[(b * a.len + t0 + tid) * a.hv + h] = 0.0f;
      }
    }
    return;
  }

  {
    RowsAhead<IO, KP, 512> k, q;
    k.load(static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h, a.sk.t, t0, Lb, a.dk, wide_qk);
    q.load(static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h, a.sq.t, t0, Lb, a.dk, wide_qk);
    k.store(sk);
    q.store(sq);
  }
  const auto at_tile = [](const bf16* s, int row, int dim) {
    float x = 0.0f;
#pragma unroll
    for (int n = N - 1; n >= 0; --n) x += float(s[n * TileK::kElems + TileK::at(row, dim)]);
    return x;
  };

  // What a slab needs, loaded while the one before it (or the last head's factors) is
  // computed: a unit or two of U, X~, dO and V a thread, and this wave's rows of S0 and E.
  constexpr int kAhead = (kC * VS / 8 + 511) / 512;
  f32x8 next_u[kAhead], next_x[kAhead], s8[VS / 32], e8[VS / 32];
  V8 next_d[kAhead], next_v[kAhead];
  const auto unit_of = [&](int n, int* row, int* unit) {
    const int u = here(tid) + 512 * n;
    *row = u / SlabV::kUnits;
    *unit = u % SlabV::kUnits;
    return u < kC * SlabV::kUnits;
  };
  const auto load_slab = [&](int hh, int v0) {
    const int h = hq * share + hh;
    const int64_t idx = (b * a.hv + h) * nchunk + c;
    const Buffer ub = buffer_of(values + idx * kC * dvp, kC * dvp * 4);
    const Buffer xb = buffer_of(xgrad + idx * kC * dvp, kC * dvp * 4);
    const Buffer db = rows_of(static_cast<const IO*>(b_.dout) + (b * a.len * a.hv + h) * a.dv + t0 * v_t, rows, v_t, a.dv);
    const Buffer vb = rows_of(static_cast<const IO*>(a.v) + b * a.sv.b + h * a.sv.h + t0 * a.sv.t, rows, a.sv.t, a.dv);
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      int row, unit;
      const bool live = unit_of(n, &row, &unit);
      const int c8 = v0 + 8 * unit, at = live && c8 < dvp ? (row * dvp + c8) * 4 : kOutside, left = live ? a.dv - c8 : 0;
      load_wide(ub, at, &next_u[n]);
      load_wide(xb, at, &next_x[n]);
      load8<IO>(db, (row * int(v_t) + c8) * int(sizeof(IO)), left, wide_d, &next_d[n]);
      load8<IO>(vb, (row * int(a.sv.t) + c8) * int(sizeof(IO)), row < rows ? left : 0, wide_v, &next_v[n]);
    }
  };
  const auto load_states = [&](int hh, int v0) {
    const int64_t idx = (b * a.hv + hq * share + hh) * nchunk + c;
    const Buffer sb = buffer_of(states + idx * KP * dvp, KP * dvp * 4);
    const Buffer eb = buffer_of(adjoints + idx * KP * dvp, KP * dvp * 4);
    const int l = here(lane), row = 16 * kt + (l & 15);
#pragma unroll
    for (int s = 0; s < VS / 32; ++s) {
      const int at = v0 + 32 * s < dvp ? (row * dvp + v0 + 32 * s + 8 * (l >> 4)) * 4 : kOutside;
      load_wide(sb, at, &s8[s]);
      load_wide(eb, at, &e8[s]);
    }
  };
  load_slab(0, 0);
  load_states(0, 0);

  f32x4 dq[MT] = {}, dk[MT] = {};
  for (int hh = 0; hh < share; ++hh) {
    const int h = hq * share + hh;
    const int i = here(lane & 15), qd = here(lane >> 4);  // LDS addresses are not kept across heads
    const int64_t idx = (b * a.hv + h) * nchunk + c;
    const Buffer gb = rows_of(static_cast<const IO*>(b_.dv) + (b * a.len * a.hv + h) * a.dv + t0 * v_t, out_rows, v_t, a.dv);
    __syncthreads();  // the last head's readers are done
    if (tid < kVecFloatsBwd) svec[tid] = vec[idx * kVecFloatsBwd + tid];
    if (tid < kC) sxv[tid] = 0.0f;
    if (wave == 7) {
      const int t = t0 + lane;
      const float g = t < Lb ? clamp_decay(a.g[b * a.sg.b + t * a.sg.t + h * a.sg.h]) : 0.0f;
      gsum[lane] = wave_running_sum(double(g));
    }

    f32x4 h1[MT] = {}, h2[MT] = {}, h3[MT] = {}, gacc[3] = {};
    float se = 0.0f;
    for (int v0 = 0; v0 < dvp; v0 += VS) {
      const bool more = v0 + VS < dvp, any = more || hh + 1 < share;
      const int next_hh = more ? hh : hh + 1, next_v0 = more ? v0 + VS : 0;
      __syncthreads();
      // the slab of U, X~ and dO; dV = beta X~ and X~ . v on the way
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        int row, unit;
        if (!unit_of(n, &row, &unit)) continue;
        const int c8 = v0 + 8 * unit, lds_at = SlabV::at(row, unit);
        const Frag<3> fu = split(next_u[n]), fx = split(next_x[n]);
        const auto fd = as_frag(next_d[n]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          *reinterpret_cast<bf16x8*>(su + k * SlabV::kElems + lds_at) = fu.t[k];
          *reinterpret_cast<bf16x8*>(sx + k * SlabV::kElems + lds_at) = fx.t[k];
        }
#pragma unroll
        for (int k = 0; k < N; ++k) *reinterpret_cast<bf16x8*>(sd + k * SlabV::kElems + lds_at) = fd.t[k];
        const float beta = svec[4 * kC + row];
        float dot = 0.0f;
        V8 y;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dot += next_x[n][j] * float(next_v[n][j]);
          y[j] = IO(row < rows ? beta * next_x[n][j] : 0.0f);  // past the row's end whatever X~ holds
        }
        store8<IO>(gb, (row * int(v_t) + c8) * int(sizeof(IO)), a.dv - c8, wide_gv, y);
#pragma unroll
        for (int k = 1; k < SlabV::kUnits; k *= 2) dot += __shfl_xor(dot, k);
        if (unit == 0) sxv[row] += dot;  // the same thread for every slab
      }
      if (any) load_slab(next_hh, next_v0);
      __syncthreads();
      // products with the states: dO S0^T, X~ S0^T, U E^T
#pragma unroll
      for (int s = 0; s < VS / 32; ++s) {
        if (v0 + 32 * s >= dvp) break;
        const Frag<3> fs = split(s8[s]), fe = split(e8[s]);
#pragma unroll
        for (int j = 0; j < 8; ++j) se += s8[s][j] * e8[s][j];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int lds_at = SlabV::at(16 * (m0 + m) + i, 4 * s + qd);
          Frag<N> fd;
          Frag<3> fx, fu;
#pragma unroll
          for (int k = 0; k < N; ++k) fd.t[k] = row_frag(sd + k * SlabV::kElems + lds_at);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            fx.t[k] = row_frag(sx + k * SlabV::kElems + lds_at);
            fu.t[k] = row_frag(su + k * SlabV::kElems + lds_at);
          }
          h1[m] = mul(fd, fs, h1[m]);
          h2[m] = mul(fx, fs, h2[m]);
          h3[m] = mul(fu, fe, h3[m]);
        }
        // dO U^T and X~ U^T, ten lower tiles each, two or three a wave
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          const int item = wave + 8 * n;
          if (item >= 20) break;
          const int tile = item < 10 ? item : item - 10;
          const int rt = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, ct = tile - rt * (rt + 1) / 2;
          const int row_at = SlabV::at(16 * rt + i, 4 * s + qd), col_at = SlabV::at(16 * ct + i, 4 * s + qd);
          Frag<3> fu;
#pragma unroll
          for (int k = 0; k < 3; ++k) fu.t[k] = row_frag(su + k * SlabV::kElems + col_at);
          if (item < 10) {
            Frag<N> fd;
#pragma unroll
            for (int k = 0; k < N; ++k) fd.t[k] = row_frag(sd + k * SlabV::kElems + row_at);
            gacc[n] = mul(fd, fu, gacc[n]);
          } else {
            Frag<3> fx;
#pragma unroll
            for (int k = 0; k < 3; ++k) fx.t[k] = row_frag(sx + k * SlabV::kElems + row_at);
            gacc[n] = mul(fx, fu, gacc[n]);
          }
        }
      }
      if (any) load_states(next_hh, next_v0);
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) se += __shfl_xor(se, m);
    if (lane == 0) sse[wave] = m0 == 0 ? se : 0.0f;  // waves of the same key tile hold the same sum
    // h1: dq, h2: -R, h3: U E^T's part of W (all times the inverse norms)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int tok = 16 * (m0 + m) + 4 * qd;
      h1[m] *= *reinterpret_cast<const f32x4*>(&svec[2 * kC + tok]);
      h2[m] *= *reinterpret_cast<const f32x4*>(&svec[tok]);
      h3[m] *= *reinterpret_cast<const f32x4*>(&svec[kC + tok]);
    }
    // the factors take the slabs' place: masked, decayed, times the inverse norms.  dO U^T
    // to g0, X~ U^T to g1, -beta X~ U^T to g2, where given
    const auto put = [&](bf16* g0, bf16* g1, bf16* g2) {
      const auto write = [&](bf16* dst, int at, float x) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const bf16 t = bf16(x);
          dst[k * kG + at] = t;
          x -= float(t);
        }
      };
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const int item = wave + 8 * n;
        if (item >= 20 || (item < 10 ? !g0 : !g1 && !g2)) continue;
        const int tile = item < 10 ? item : item - 10;
        const int rt = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, ct = tile - rt * (rt + 1) / 2;
        const int tj = 16 * ct + i, row = 16 * rt + 4 * qd;
        const double sum_j = gsum[tj];
        const float rk_j = svec[5 * kC + tj];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ti = row + r, at = ti * kLdG + tj;
          const float x = gacc[n][r] * expf(float(gsum[ti] - sum_j)) * rk_j;
          if (item < 10) {
            write(g0, at, tj <= ti ? x * (a.scale * svec[6 * kC + ti]) : 0.0f);
          } else {
            const float y = tj < ti ? x * svec[5 * kC + ti] : 0.0f;
            if (g1) write(g1, at, y);
            if (g2) write(g2, at, -y * svec[4 * kC + ti]);
          }
        }
      }
      if (wave >= 6) {  // tiles (0, 1) and (2, 3): above the diagonal, but in the fragments read
        const int at = ((wave - 6) * 32 + 4 * qd) * kLdG + (wave - 6) * 32 + 16 + i;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (g0) write(g0, at + r * kLdG, 0.0f);
          if (g1) write(g1, at + r * kLdG, 0.0f);
          if (g2) write(g2, at + r * kLdG, 0.0f);
        }
      }
    };
    f32x4 w[MT] = {};
    // acc += G B over tokens j <= i, and acc += G^T B over i >= j
    const auto by_rows = [&](f32x4 (&acc)[MT], const bf16* g, const bf16* tile) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (m0 + m < 2 && s == 1) continue;
          Frag<3> fg;
#pragma unroll
          for (int n = 0; n < 3; ++n) fg.t[n] = row_frag(g + n * kG + (16 * (m0 + m) + i) * kLdG + 32 * s + 8 * qd);
          Frag<N> fb;
#pragma unroll
          for (int t = 0; t < N; ++t) fb.t[t] = col_frag<KP>(tile + t * TileK::kElems, 32 * s + 8 * qd, 16 * kt + 4 * (i & 3));
          acc[m] = mul(fg, fb, acc[m]);
        }
    };
    const auto by_cols = [&](f32x4 (&acc)[MT], const bf16* g, const bf16* tile) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (m0 + m >= 2 && s == 0) continue;
          Frag<3> fg;
#pragma unroll
          for (int n = 0; n < 3; ++n)
            fg.t[n] = col_frag(g + n * kG + (32 * s + 8 * qd + (i >> 2)) * kLdG + 16 * (m0 + m) + 4 * (i & 3), kLdG);
          Frag<N> fb;
#pragma unroll
          for (int t = 0; t < N; ++t) fb.t[t] = col_frag<KP>(tile + t * TileK::kElems, 32 * s + 8 * qd, 16 * kt + 4 * (i & 3));
          acc[m] = mul(fg, fb, acc[m]);
        }
    };
    __syncthreads();
    if constexpr (Lds::kFactors == 3) {
      put(shared, shared + 3 * kG, shared + 6 * kG);
      __syncthreads();
      by_rows(h1, shared, sk);
      by_rows(h2, shared + 3 * kG, sk);
      by_cols(w, shared, sq);
      by_cols(w, shared + 6 * kG, sk);
    } else {
      put(shared, nullptr, nullptr);
      __syncthreads();
      by_rows(h1, shared, sk);
      by_cols(w, shared, sq);
      __syncthreads();
      put(nullptr, shared, nullptr);
      __syncthreads();
      by_rows(h2, shared, sk);
      __syncthreads();
      put(nullptr, nullptr, shared);
      __syncthreads();
      by_cols(w, shared, sk);
    }

    // per token: q . dq, k . R, k . (W without U E^T), k . U E^T
    const int sum_tok = 16 * m0 + 16 * ((i >> 2) % MT) + 4 * qd + (i & 3);  // value i of the sums
    const auto dots = [&](int which, auto value) {
      float v[4 * MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[4 * m + r] = value(m, r, 16 * (m0 + m) + 4 * qd + r);
      sdot[kt][which][sum_tok] = lane_sums(v);
      __builtin_amdgcn_sched_barrier(0);  // one set of sums in registers at a time
    };
    const int dim = 16 * kt + i;
    dots(0, [&](int m, int r, int tok) { return at_tile(sq, tok, dim) * h1[m][r]; });
    dots(1, [&](int m, int r, int tok) { return -at_tile(sk, tok, dim) * h2[m][r]; });
    dots(2, [&](int m, int r, int tok) { return at_tile(sk, tok, dim) * w[m][r]; });
    dots(3, [&](int m, int r, int tok) { return at_tile(sk, tok, dim) * h3[m][r]; });
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      dq[m] += h1[m];
      dk[m] += w[m] + h3[m] - *reinterpret_cast<const f32x4*>(&svec[4 * kC + 16 * (m0 + m) + 4 * qd]) * h2[m];
    }
    __syncthreads();
    if (wave == 0) {
      const int t = t0 + lane;
      float d[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        d[x] = sdot[0][x][lane];
#pragma unroll
        for (int k = 1; k < kTilesK; ++k) d[x] += sdot[k][x][lane];
      }
      const float beta = svec[4 * kC + lane];
      const double own = double(d[0]) + double(beta) * d[1] - d[2];
      // sum over i >= t of own, over j < t of k . U E^T, and exp(G_C) <E, S0>
      const double upto = wave_running_sum(own), wrote = wave_running_sum(double(d[3]));
      const double all = lane_of(upto, 63);
      double s0e = 0.0;
#pragma unroll
      for (int k = 0; k < 8; ++k) s0e += sse[k];
      if (t < L) {
        const int64_t at = (b * a.len + t) * a.hv + h;
        b_.dg[at] = t < Lb ? float((all - upto + own) + (wrote - d[3]) + svec[3 * kC] * s0e) : 0.0f;
        b_.dbeta[at] = t < Lb ? sxv[lane] + d[1] : 0.0f;
      }
    }
  }

  // through the norms: d raw = d - raw r^2 (raw . d), d already times r
  __syncthreads();
  if (a.qk_norm) {
    float dots_q[4 * MT], dots_k[4 * MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tok = 16 * (m0 + m) + 4 * qd + r, dim = 16 * kt + i;
        dots_q[4 * m + r] = at_tile(sq, tok, dim) * dq[m][r];
        dots_k[4 * m + r] = at_tile(sk, tok, dim) * dk[m][r];
      }
    const int sum_tok = 16 * m0 + 16 * ((i >> 2) % MT) + 4 * qd + (i & 3);
    sdot[kt][0][sum_tok] = lane_sums(dots_q);
    sdot[kt][1][sum_tok] = lane_sums(dots_k);
    __syncthreads();
  }
  const int dim = 16 * kt + i;
  const Buffer dqb = rows_of(dq_out + t0 * qk_t, out_rows, qk_t, a.dk), dkb = rows_of(dk_out + t0 * qk_t, out_rows, qk_t, a.dk);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = 16 * (m0 + m) + 4 * qd + r;
      float fq = 0.0f, fk = 0.0f;
      if (a.qk_norm) {
        const float rk = svec[5 * kC + tok], rq = svec[6 * kC + tok];
#pragma unroll
        for (int k = 0; k < kTilesK; ++k) {
          fq += sdot[k][0][tok];
          fk += sdot[k][1][tok];
        }
        fq *= rq * rq;
        fk *= rk * rk;
      }
      const int at = dim < a.dk ? (tok * int(qk_t) + dim) * int(sizeof(IO)) : kOutside;
      store1(dqb, at, IO(tok < rows ? dq[m][r] - fq * at_tile(sq, tok, dim) : 0.0f));
      store1(dkb, at, IO(tok < rows ? dk[m][r] - fk * at_tile(sk, tok, dim) : 0.0f));
    }
}

// Value columns of a slab: what LDS holds beside K and Q.
template <typename IO, int KP>
void launch_grad(const DeltaBwdArgs& b, int n, const float* vec, const float* s, const float* e, const float* u,
                 const float* x, int dvp, int wide, hipStream_t stream) {
  constexpr bool kBf16 = std::is_same<IO, bf16>::value;
  constexpr int kMost = kBf16 || KP == 64 ? 64 : 32;
  const dim3 grid{unsigned(b.f.batch * b.f.hk * n)};
  delta_grad_kernel<IO, KP, kMost><<<grid, 512, 0, stream>>>(b, n, vec, s, e, u, x, dvp, wide);
}

template <typename IO, int KP, int W>
hipError_t launch_bwd(const DeltaBwdArgs& b, const DeltaBwdPlan& p, char* ws, hipStream_t stream) {
  const DeltaArgs& a = b.f;
  int wide = wide_flags<IO>(a) & ~4;
  if (a.dv % 8 == 0 && reinterpret_cast<uintptr_t>(b.dout) % 16 == 0) wide |= 4;
  if (a.dv % 8 == 0 && reinterpret_cast<uintptr_t>(b.dv) % 16 == 0) wide |= 16;
  const DeltaPlan& f = p.f;
  const int n = int(f.nchunk), nvb = (f.dvp + 16 * W - 1) / (16 * W);
  const auto floats = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  char *ft = ws + f.off_t, *ftt = ws + p.off_tt, *fpt = ws + p.off_pt;
  float *vec = floats(f.off_vec), *u = floats(p.off_u), *x = floats(p.off_y), *s = floats(p.off_s),
        *e = floats(p.off_ds), *ends = floats(f.off_ends), *moves = floats(f.off_moves), *back = floats(p.off_back);
  const WalkArgs w{n, nvb, f.nseg, f.seg_chunks, f.dvp, wide, ft, nullptr, vec, s, u, ends, moves};
  const WalkBackArgs wb{n, nvb, f.nseg, f.seg_chunks, f.dvp, wide, ftt, fpt, vec, e, x, back};
  const int64_t bh = a.batch * a.hv;
  const dim3 walk{unsigned(bh * f.nseg * nvb)}, chain{unsigned(bh * (f.dvp / 16))};
  if (n > 0) {
    delta_prep_kernel<IO, KP, true><<<dim3(unsigned(bh * n)), 256, 0, stream>>>(a, n, ft, fpt, ftt, vec, wide);
    if (f.nseg > 1) {
      constexpr int kIdent = (KP + 16 * W - 1) / (16 * W);
      delta_chunk_kernel<IO, KP, W, kEnds>
          <<<dim3(unsigned(bh * f.nseg * (nvb + kIdent))), 64 * W, 0, stream>>>(a, w, kVecFloatsBwd);
      delta_chunk_bwd_kernel<IO, KP, W, true><<<walk, 64 * W, 0, stream>>>(b, wb);
    }
    if (f.nseg > 2) {
      delta_carry_kernel<KP, false><<<chain, 2 * KP, 0, stream>>>(moves, ends, f.nseg, f.dvp);
      delta_carry_kernel<KP, true><<<chain, 2 * KP, 0, stream>>>(moves, back, f.nseg, f.dvp);
    }
    delta_chunk_kernel<IO, KP, W, kStates><<<walk, 64 * W, 0, stream>>>(a, w, kVecFloatsBwd);
  }
  delta_chunk_bwd_kernel<IO, KP, W, false><<<walk, 64 * W, 0, stream>>>(b, wb);
  if (n > 0)
    launch_grad<IO, KP>(b, n, vec, s, e, u, x, f.dvp, wide, stream);
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_bwd(const DeltaBwdArgs& b, const DeltaBwdPlan& p, char* ws, hipStream_t stream) {
  if constexpr (std::is_same<IO, bf16>::value)  // float32 walks have four waves
    if (p.f.waves == 8)
      return p.f.kp == 64 ? launch_bwd<IO, 64, 8>(b, p, ws, stream) : launch_bwd<IO, 128, 8>(b, p, ws, stream);
  return p.f.kp == 64 ? launch_bwd<IO, 64, 4>(b, p, ws, stream) : launch_bwd<IO, 128, 4>(b, p, ws, stream);
}

}  // namespace delta

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

DeltaBwdPlan make_delta_bwd_plan(int64_t batch, int64_t len, int hk, int hv, int dk, int dv, bool io_bf16) {
  DeltaBwdPlan p{};
  p.f = make_delta_plan(batch, len, hk, hv, dk, dv, io_bf16);
  if (p.f.recurrent) {  // the gradients always go by chunks, and these rows have at most one
    p.f.recurrent = 0;
    p.f.nseg = p.f.seg_chunks = 1;
  }
  const size_t n = size_t(batch) * size_t(hv) * size_t(p.f.nchunk), segs = size_t(batch) * size_t(hv) * size_t(p.f.nseg);
  const size_t kp = size_t(p.f.kp), dvp = size_t(p.f.dvp);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t off = at;
    at += round256(bytes);
    return off;
  };
  p.f.off_t = take(n * delta::kFrags * 3 * delta::kFragBytes);
  p.off_tt = take(n * delta::kFrags * 3 * delta::kFragBytes);
  p.off_pt = take(n * delta::kFrags * 3 * delta::kFragBytes);
  p.f.off_vec = take(n * delta::kVecFloatsBwd * 4);
  p.off_u = take(n * kDeltaChunk * dvp * 4);
  p.off_y = take(n * kDeltaChunk * dvp * 4);
  p.off_s = take(n * kp * dvp * 4);
  p.off_ds = take(n * kp * dvp * 4);
  const bool split = p.f.nseg > 1;
  p.f.off_ends = take(split ? segs * kp * dvp * 4 : 0);
  p.f.off_moves = take(split ? segs * kp * kp * 4 : 0);
  p.off_back = take(split ? segs * kp * dvp * 4 : 0);
  p.workspace_bytes = at;
  return p;
}

hipError_t launch_delta_bwd(const DeltaBwdArgs& b, const DeltaBwdPlan& p, char* ws, hipStream_t stream) {
  return b.f.io_bf16 ? delta::launch_bwd<delta::bf16>(b, p, ws, stream) : delta::launch_bwd<float>(b, p, ws, stream);
}

}  // namespace sscan
