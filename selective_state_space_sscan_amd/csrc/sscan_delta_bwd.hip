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
// the forward walk's, transposed.
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
  typedef WalkLds<IO, KP, true, 3, kVecs> Lds;
  __shared__ __attribute__((aligned(256))) char lds[Lds::kSets * Lds::kSet];

  const DeltaArgs& a = b_.f;
  const int tid = int(threadIdx.x), lane = tid & 63, wave = wave_id(), i = lane & 15, qd = lane >> 4;
  const int vb = int(blockIdx.x % unsigned(w.nvb)), seg = int(blockIdx.x / unsigned(w.nvb) % unsigned(w.nseg));
  const int64_t bh = blockIdx.x / unsigned(w.nvb) / unsigned(w.nseg), b = bh / a.hv, at_seg = bh * w.nseg + seg;
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

__device__ __forceinline__ float row16_sum(float x) {
#pragma unroll
  for (int m = 1; m < 16; m *= 2) x += __shfl_xor(x, m);
  return x;
}

// One block per (batch row, key head, chunk); the value heads that share the key head
// are walked in order and their dq, dk summed in registers.  Wave w owns the key
// dimensions of tiles w, w + 4 for all 64 tokens.
template <typename IO, int KP>
__global__ __launch_bounds__(256) void delta_grad_kernel(DeltaBwdArgs b_, int nchunk, const float* vec,
                                                         const float* states, const float* adjoints,
                                                         const float* values, const float* xgrad, int dvp, int wide) {
  constexpr int N = Io<IO>::kN, NT = KP / 64, kLdG = 72;
  typedef Tile<KP> TileK;
  typedef typename Io<IO>::V8 V8;
  __shared__ __attribute__((aligned(16))) bf16 sk[N][TileK::kElems];
  __shared__ __attribute__((aligned(16))) bf16 sq[N][TileK::kElems];
  __shared__ __attribute__((aligned(16))) bf16 sg[3][kC * kLdG];
  __shared__ __attribute__((aligned(16))) float svec[kVecFloatsBwd];
  __shared__ double gsum[kC];
  __shared__ float sdot[4][4][kC], sxv[kC], sse[4];

  const DeltaArgs& a = b_.f;
  const int tid = int(threadIdx.x), lane = tid & 63, wave = wave_id(), i = lane & 15, qd = lane >> 4;
  const int c = int(blockIdx.x % unsigned(nchunk));
  const int64_t bhk = blockIdx.x / unsigned(nchunk), b = bhk / a.hk;
  const int hq = int(bhk % a.hk), share = a.hv / a.hk;
  const int L = int(a.len), Lb = row_len(a.lengths, b, a.len), t0 = c * kC;
  const int64_t qk_t = int64_t(a.hk) * a.dk, v_t = int64_t(a.hv) * a.dv;
  const bool wide_qk = wide & 1, wide_v = wide & 2, wide_d = wide & 4, wide_gv = wide & 16;
  IO* dq_out = static_cast<IO*>(b_.dq) + (b * a.len * a.hk + hq) * a.dk;
  IO* dk_out = static_cast<IO*>(b_.dk) + (b * a.len * a.hk + hq) * a.dk;

  if (t0 >= Lb) {  // past the row's length: zeros
    const int rows = L - t0 < kC ? L - t0 : kC;
    for (int u = tid; u < rows * a.dk; u += 256) {
      const int64_t at = (t0 + u / a.dk) * qk_t + u % a.dk;
      dq_out[at] = IO(0.0f);
      dk_out[at] = IO(0.0f);
    }
    for (int hh = 0; hh < share; ++hh) {
      const int64_t h = hq * share + hh;
      IO* dv_out = static_cast<IO*>(b_.dv) + (b * a.len * a.hv + h) * a.dv;
      for (int u = tid; u < rows * a.dv; u += 256) dv_out[(t0 + u / a.dv) * v_t + u % a.dv] = IO(0.0f);
      if (tid < rows) {
        b_.dg[(b * a.len + t0 + tid) * a.hv + h] = 0.0f;
        b_.dbeta[(b * a.len + t0 + tid) * a.hv + h] = 0.0f;
      }
    }
    return;
  }

  const IO* kp = static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h;
  const IO* qp = static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h;
  for (int u = tid; u < kC * KP / 8; u += 256) {
    const int row = u / (KP / 8), d8 = (u % (KP / 8)) * 8;
    const bool in = t0 + row < Lb;
    const auto fk = as_frag(load8(kp + (t0 + row) * a.sk.t + d8, in ? a.dk - d8 : 0, wide_qk));
    const auto fq = as_frag(load8(qp + (t0 + row) * a.sq.t + d8, in ? a.dk - d8 : 0, wide_qk));
#pragma unroll
    for (int n = 0; n < N; ++n) {
      *reinterpret_cast<bf16x8*>(&sk[n][TileK::unit_at(row, d8 / 8)]) = fk.t[n];
      *reinterpret_cast<bf16x8*>(&sq[n][TileK::unit_at(row, d8 / 8)]) = fq.t[n];
    }
  }
  const auto at_tile = [](const bf16 (&s)[N][TileK::kElems], int row, int dim) {
    float x = 0.0f;
#pragma unroll
    for (int n = N - 1; n >= 0; --n) x += float(s[n][TileK::at(row, dim)]);
    return x;
  };

  f32x4 dq[4][NT] = {}, dk[4][NT] = {};
  for (int hh = 0; hh < share; ++hh) {
    const int h = hq * share + hh;
    const int64_t idx = (b * a.hv + h) * nchunk + c;
    const float* up = values + idx * kC * dvp;
    const float* xp = xgrad + idx * kC * dvp;
    const float* sp = states + idx * KP * dvp;
    const float* ep = adjoints + idx * KP * dvp;
    const IO* dp = static_cast<const IO*>(b_.dout) + (b * a.len * a.hv + h) * a.dv;
    __syncthreads();
    for (int u = tid; u < kVecFloatsBwd; u += 256) svec[u] = vec[idx * kVecFloatsBwd + u];
    if (wave == 0) {
      const int t = t0 + lane;
      const float g = t < Lb ? clamp_decay(a.g[b * a.sg.b + t * a.sg.t + h * a.sg.h]) : 0.0f;
      gsum[lane] = wave_running_sum(double(g));
    }
    __syncthreads();

    // dv = beta x~, and x~ . v per token (four threads a token)
    {
      const int row = tid >> 2, t = t0 + row;
      const float beta = svec[4 * kC + row];
      const IO* vp = static_cast<const IO*>(a.v) + b * a.sv.b + t * a.sv.t + h * a.sv.h;
      IO* dst = static_cast<IO*>(b_.dv) + ((b * a.len + t) * a.hv + h) * a.dv;
      float dot = 0.0f;
      if (t < L)
        for (int c8 = (tid & 3) * 8; c8 < a.dv; c8 += 32) {
          const f32x8 x = load8(xp + row * dvp + c8, 8, true);
          const V8 v = load8(vp + c8, t < Lb ? a.dv - c8 : 0, wide_v);
          V8 y;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dot += x[j] * float(v[j]);
            y[j] = IO(beta * x[j]);
          }
          if (wide_gv) {
            *reinterpret_cast<V8*>(dst + c8) = y;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c8 + j < a.dv) dst[c8 + j] = y[j];
          }
        }
      dot += __shfl_xor(dot, 1);
      dot += __shfl_xor(dot, 2);
      if ((tid & 3) == 0) sxv[row] = dot;
    }

    // dO U^T and X~ U^T: wave w takes tokens 16 w .. + 15 against all earlier ones
    f32x4 g1[4] = {}, g2[4] = {};
    {
      const int t = t0 + 16 * wave + i;
      for (int v0 = 0; v0 < dvp; v0 += 32) {
        const int v8 = v0 + 8 * qd;
        const auto fd = as_frag(load8(dp + t * v_t + v8, t < Lb ? a.dv - v8 : 0, wide_d));
        const Frag<3> fx = split(load8(xp + (16 * wave + i) * dvp + v8, 8, true));
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)
          if (ct <= wave) {
            const Frag<3> fu = split(load8(up + (16 * ct + i) * dvp + v8, 8, true));
            g1[ct] = mul(fd, fu, g1[ct]);
            g2[ct] = mul(fx, fu, g2[ct]);
          }
      }
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ti = 16 * wave + 4 * qd + r, tj = 16 * ct + i;
          const float decay = tj <= ti ? expf(float(gsum[ti] - gsum[tj])) * svec[5 * kC + tj] : 0.0f;
          g1[ct][r] = tj <= ti ? g1[ct][r] * decay * a.scale * svec[6 * kC + ti] : 0.0f;
          g2[ct][r] = tj < ti ? g2[ct][r] * decay * svec[5 * kC + ti] : 0.0f;
        }
    }
    const auto put = [&](const f32x4 (&g)[4], bool with_beta) {
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ti = 16 * wave + 4 * qd + r;
          float x = with_beta ? g[ct][r] * svec[4 * kC + ti] : g[ct][r];
#pragma unroll
          for (int n = 0; n < 3; ++n) {
            const bf16 t = bf16(x);
            sg[n][ti * kLdG + 16 * ct + i] = t;
            x -= float(t);
          }
        }
    };
    put(g1, false);

    // products with the states: dO S0^T, X~ S0^T, U E^T
    f32x4 h1[4][NT] = {}, h2[4][NT] = {}, h3[4][NT] = {};
    float se = 0.0f;
    for (int v0 = 0; v0 < dvp; v0 += 32) {
      const int v8 = v0 + 8 * qd;
      Frag<3> fs[NT], fe[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int dim = 16 * (wave + 4 * n) + i;
        const f32x8 s = load8(sp + dim * dvp + v8, 8, true), e = load8(ep + dim * dvp + v8, 8, true);
        fs[n] = split(s);
        fe[n] = split(e);
#pragma unroll
        for (int j = 0; j < 8; ++j) se += s[j] * e[j];
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int row = 16 * m + i, t = t0 + row;
        const auto fd = as_frag(load8(dp + t * v_t + v8, t < Lb ? a.dv - v8 : 0, wide_d));
        const Frag<3> fx = split(load8(xp + row * dvp + v8, 8, true));
        const Frag<3> fu = split(load8(up + row * dvp + v8, 8, true));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          h1[m][n] = mul(fd, fs[n], h1[m][n]);
          h2[m][n] = mul(fx, fs[n], h2[m][n]);
          h3[m][n] = mul(fu, fe[n], h3[m][n]);
        }
      }
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) se += __shfl_xor(se, m);
    if (lane == 0) sse[wave] = se;
    // h1: dq, h2: -R, h3: U E^T's part of W (all times the inverse norms)
    float kh3[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int tok = 16 * m + 4 * qd;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        kh3[m][r] = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          h1[m][n][r] *= svec[2 * kC + tok + r];
          h2[m][n][r] *= svec[tok + r];
          h3[m][n][r] *= svec[kC + tok + r];
          kh3[m][r] += at_tile(sk, tok + r, 16 * (wave + 4 * n) + i) * h3[m][n][r];
        }
      }
    }
    f32x4 w[4][NT] = {};
    // lower: acc += G B over tokens j <= i; upper: acc += G^T B over i >= j
    const auto by_rows = [&](f32x4 (&acc)[4][NT], const bf16 (&tile)[N][TileK::kElems]) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (lower_frag(m, s) < 0) continue;
          Frag<3> fg;
#pragma unroll
          for (int n = 0; n < 3; ++n) fg.t[n] = row_frag(&sg[n][(16 * m + i) * kLdG + 32 * s + 8 * qd]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            Frag<N> fb;
#pragma unroll
            for (int t = 0; t < N; ++t)
              fb.t[t] = col_frag<KP>(tile[t], 32 * s + 8 * qd, 16 * (wave + 4 * n) + 4 * (i & 3));
            acc[m][n] = mul(fg, fb, acc[m][n]);
          }
        }
    };
    const auto by_cols = [&](f32x4 (&acc)[4][NT], const bf16 (&tile)[N][TileK::kElems], bool minus) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (upper_frag(m, s) < 0) continue;
          Frag<3> fg;
#pragma unroll
          for (int n = 0; n < 3; ++n) {
            fg.t[n] = col_frag(&sg[n][(32 * s + 8 * qd + (i >> 2)) * kLdG + 16 * m + 4 * (i & 3)], kLdG);
            if (minus) fg.t[n] = -fg.t[n];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            Frag<N> fb;
#pragma unroll
            for (int t = 0; t < N; ++t)
              fb.t[t] = col_frag<KP>(tile[t], 32 * s + 8 * qd, 16 * (wave + 4 * n) + 4 * (i & 3));
            acc[m][n] = mul(fg, fb, acc[m][n]);
          }
        }
    };
    __syncthreads();
    by_rows(h1, sk);
    by_cols(w, sq, false);
    __syncthreads();
    put(g2, false);
    __syncthreads();
    by_rows(h2, sk);
    __syncthreads();
    put(g2, true);
    __syncthreads();
    by_cols(w, sk, true);

    // per token: q . dq, k . R, k . (W without U E^T), k . U E^T
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tok = 16 * m + 4 * qd + r;
        const float beta = svec[4 * kC + tok];
        float d[4] = {0.0f, 0.0f, 0.0f, kh3[m][r]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int dim = 16 * (wave + 4 * n) + i;
          const float k = at_tile(sk, tok, dim), q = at_tile(sq, tok, dim);
          d[0] += q * h1[m][n][r];
          d[1] -= k * h2[m][n][r];
          d[2] += k * w[m][n][r];
          dq[m][n][r] += h1[m][n][r];
          dk[m][n][r] += w[m][n][r] + h3[m][n][r] - beta * h2[m][n][r];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          d[x] = row16_sum(d[x]);
          if (i == 0) sdot[wave][x][tok] = d[x];
        }
      }
    __syncthreads();
    if (wave == 0) {
      const int t = t0 + lane;
      float d[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) d[x] = (sdot[0][x][lane] + sdot[1][x][lane]) + (sdot[2][x][lane] + sdot[3][x][lane]);
      const float beta = svec[4 * kC + lane];
      const double own = double(d[0]) + double(beta) * d[1] - d[2];
      // sum over i >= t of own, over j < t of k . U E^T, and exp(G_C) <E, S0>
      const double upto = wave_running_sum(own), wrote = wave_running_sum(double(d[3]));
      const double all = __shfl(upto, 63);
      const double s0e = double(sse[0]) + sse[1] + sse[2] + sse[3];
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
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tok = 16 * m + 4 * qd + r;
        float d[2] = {};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int dim = 16 * (wave + 4 * n) + i;
          d[0] += at_tile(sq, tok, dim) * dq[m][n][r];
          d[1] += at_tile(sk, tok, dim) * dk[m][n][r];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          d[x] = row16_sum(d[x]);
          if (i == 0) sdot[wave][x][tok] = d[x];
        }
      }
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = 16 * m + 4 * qd + r, t = t0 + tok;
      float fq = 0.0f, fk = 0.0f;
      if (a.qk_norm) {
        const float rk = svec[5 * kC + tok], rq = svec[6 * kC + tok];
        fq = rq * rq * ((sdot[0][0][tok] + sdot[1][0][tok]) + (sdot[2][0][tok] + sdot[3][0][tok]));
        fk = rk * rk * ((sdot[0][1][tok] + sdot[1][1][tok]) + (sdot[2][1][tok] + sdot[3][1][tok]));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int dim = 16 * (wave + 4 * n) + i;
        if (t < L && dim < a.dk) {
          dq_out[t * qk_t + dim] = IO(dq[m][n][r] - fq * at_tile(sq, tok, dim));
          dk_out[t * qk_t + dim] = IO(dk[m][n][r] - fk * at_tile(sk, tok, dim));
        }
      }
    }
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
  const dim3 walk{unsigned(bh * f.nseg * nvb)}, chain{unsigned(bh * ((f.dvp + 63) / 64))};
  if (n > 0) {
    delta_prep_kernel<IO, KP, true><<<dim3(unsigned(bh * n)), 256, 0, stream>>>(a, n, ft, fpt, ftt, vec, wide);
    if (f.nseg > 1) {
      constexpr int kIdent = (KP + 16 * W - 1) / (16 * W);
      delta_chunk_kernel<IO, KP, W, kEnds>
          <<<dim3(unsigned(bh * f.nseg * (nvb + kIdent))), 64 * W, 0, stream>>>(a, w, kVecFloatsBwd);
      delta_chunk_bwd_kernel<IO, KP, W, true><<<walk, 64 * W, 0, stream>>>(b, wb);
    }
    if (f.nseg > 2) {
      delta_carry_kernel<KP, 4, false><<<chain, 256, 0, stream>>>(moves, ends, f.nseg, f.dvp, (f.dvp + 63) / 64);
      delta_carry_kernel<KP, 4, true><<<chain, 256, 0, stream>>>(moves, back, f.nseg, f.dvp, (f.dvp + 63) / 64);
    }
    delta_chunk_kernel<IO, KP, W, kStates><<<walk, 64 * W, 0, stream>>>(a, w, kVecFloatsBwd);
  }
  delta_chunk_bwd_kernel<IO, KP, W, false><<<walk, 64 * W, 0, stream>>>(b, wb);
  if (n > 0)
    delta_grad_kernel<IO, KP><<<dim3(unsigned(a.batch * a.hk * n)), 256, 0, stream>>>(b, n, vec, s, e, u, x, f.dvp, wide);
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_bwd(const DeltaBwdArgs& b, const DeltaBwdPlan& p, char* ws, hipStream_t stream) {
  if (p.f.kp == 64)
    return p.f.waves == 8 ? launch_bwd<IO, 64, 8>(b, p, ws, stream) : launch_bwd<IO, 64, 4>(b, p, ws, stream);
  return p.f.waves == 8 ? launch_bwd<IO, 128, 8>(b, p, ws, stream) : launch_bwd<IO, 128, 4>(b, p, ws, stream);
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
