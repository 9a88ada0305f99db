// sscan_delta_chunk.h -- the gated delta rule's walk over chunks, shared by the forward
// pass and by the recomputation of the states in the backward pass.
#pragma once

#include "sscan_delta.h"
#include "sscan_delta_device.h"

namespace sscan {
namespace delta {

// A chunk's rows of K (or Q) on their way from memory to the LDS tile: loaded into
// registers while the chunk before is computed.
template <typename IO, int KP>
struct RowsAhead {
  static constexpr int kUnits = kC * KP / 8 / 256;
  typename Io<IO>::V8 x[kUnits];

  __device__ __forceinline__ void load(const IO* p, int64_t stride, int t0, int len, int dk, bool wide) {
    const Buffer rows = rows_of(p + t0 * stride, len - t0 < kC ? len - t0 : kC, stride, dk);
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int u = int(threadIdx.x) + 256 * n, row = u / (KP / 8), d8 = (u % (KP / 8)) * 8;
      load8<IO>(rows, (row * int(stride) + d8) * int(sizeof(IO)), dk - d8, wide, &x[n]);
    }
  }

  template <int N>
  __device__ __forceinline__ void store(bf16 (&tile)[N][Tile<KP>::kElems]) const {
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int u = int(threadIdx.x) + 256 * n, row = u / (KP / 8), d8 = (u % (KP / 8)) * 8;
      const auto f = as_frag(x[n]);
#pragma unroll
      for (int k = 0; k < N; ++k) *reinterpret_cast<bf16x8*>(&tile[k][row * Tile<KP>::kLd + d8]) = f.t[k];
    }
  }
};

// A contiguous block of kBytes, likewise.
template <int kBytes>
struct BytesAhead {
  static constexpr int kUnits = (kBytes / 16 + 255) / 256;
  u32x4 x[kUnits];

  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int u = int(threadIdx.x) + 256 * n;
      if (u < kBytes / 16) x[n] = reinterpret_cast<const u32x4*>(p)[u];
    }
  }

  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int u = int(threadIdx.x) + 256 * n;
      if (u < kBytes / 16) reinterpret_cast<u32x4*>(lds)[u] = x[n];
    }
  }
};

// A wave owns sixteen columns of S for the whole sequence (KP x 16, in the accumulator
// layout) and walks the chunks in order; columns are independent, so waves never
// exchange data: every product's result is the next product's B factor in the same
// lane.  A block is four waves (64 columns) that share the chunk's K and Q tiles and
// the fragments of T and P through LDS; the next chunk's are loaded into registers
// while a chunk is computed.  V and the output move between memory and the lanes that
// own them (32-byte runs of a row that the block's four waves complete to a line).
// STATES: the backward pass's recomputation, which leaves every chunk's entry state
// [KP][dvp] and U [64][dvp] in float32 instead of the output and the last state.
template <typename IO, int KP, bool STATES>
__global__ __launch_bounds__(256) void delta_chunk_kernel(DeltaArgs a, int nchunk, int nvb, const char* frag_t,
                                                          const char* frag_p, const float* vec, float* states,
                                                          float* values, int dvp, int wide) {
  constexpr int N = Io<IO>::kN, NO = Io<IO>::kOutTerms;
  constexpr int kTiles = KP / 16, kSteps = KP / 32, kVecs = STATES ? kVecFloatsBwd : kVecFloats;
  constexpr int kBytesT = kFrags * 3 * kFragBytes, kBytesP = STATES ? 16 : kFrags * NO * kFragBytes;
  typedef Tile<KP> TileK;
  __shared__ __attribute__((aligned(16))) bf16 sk[N][TileK::kElems];
  __shared__ __attribute__((aligned(16))) bf16 sq[STATES ? 1 : N][STATES ? 8 : TileK::kElems];
  __shared__ __attribute__((aligned(16))) char st[kBytesT];
  __shared__ __attribute__((aligned(16))) char sp[kBytesP];
  __shared__ __attribute__((aligned(16))) float svec[kVecFloats];

  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6, i = lane & 15, qd = lane >> 4;
  const int64_t bh = int64_t(blockIdx.x) / nvb, b = bh / a.hv;
  const int h = int(bh % a.hv), hq = h / (a.hv / a.hk);
  const int col = int(int64_t(blockIdx.x) % nvb) * 64 + 16 * wave + i;
  const int L = int(a.len), Lb = row_len(a.lengths, b, a.len);
  const int live_chunks = (Lb + kC - 1) / kC;
  const IO* kp = static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h;
  const IO* qp = static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h;
  const IO* vp = static_cast<const IO*>(a.v) + b * a.sv.b + h * a.sv.h;
  IO* op = static_cast<IO*>(a.out) + (b * a.len * a.hv + h) * a.dv;
  const int64_t out_t = int64_t(a.hv) * a.dv;
  const bool wide_qk = wide & 1, live_col = col < a.dv;
  // byte offset of this lane's first token (8 qd) and column in a chunk's rows, and the
  // rows from there to token 32 (m >> 1) + 4 (m & 1) + r
  const int v_lane = (8 * qd * int(a.sv.t) + col) * int(sizeof(IO)), v_row = int(a.sv.t) * int(sizeof(IO));
  const int o_lane = (8 * qd * int(out_t) + col) * int(sizeof(IO)), o_row = int(out_t) * int(sizeof(IO));

  f32x4 S[kTiles];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int dim = chained(m, 4 * qd + r);
      S[m][r] = (a.h0 && dim < a.dk && live_col) ? a.h0[(bh * a.dk + dim) * a.dv + col] : 0.0f;
    }

  RowsAhead<IO, KP> next_k, next_q;
  BytesAhead<kBytesT> next_t;
  BytesAhead<kBytesP> next_p;
  IO next_v[4][4];
  float next_vec = 0.0f;
  const auto load_ahead = [&](int c) {
    const int64_t idx = bh * nchunk + c;
    const int t0 = c * kC;
    next_k.load(kp, a.sk.t, t0, Lb, a.dk, wide_qk);
    next_t.load(frag_t + idx * kBytesT);
    if constexpr (!STATES) {
      next_q.load(qp, a.sq.t, t0, Lb, a.dk, wide_qk);
      next_p.load(frag_p + idx * kBytesP);
    }
    next_vec = vec[idx * kVecs + tid];
    const Buffer rows = rows_of(vp + t0 * a.sv.t, Lb - t0 < kC ? Lb - t0 : kC, a.sv.t, a.dv);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        load1(rows, live_col ? v_lane + (32 * (m >> 1) + 4 * (m & 1) + r) * v_row : kOutside, &next_v[m][r]);
  };
  if (live_chunks > 0) load_ahead(0);

  for (int c = 0; c < live_chunks; ++c) {
    const int t0 = c * kC;
    const int64_t idx = bh * nchunk + c;
    __syncthreads();  // the last chunk's readers of the tiles are done
    next_k.store(sk);
    next_t.store(st);
    if constexpr (!STATES) {
      next_q.store(sq);
      next_p.store(sp);
    }
    svec[tid] = next_vec;
    f32x4 x[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) x[m][r] = to_f32(next_v[m][r]);
    __syncthreads();
    if (c + 1 < live_chunks) load_ahead(c + 1);
    if (STATES && col < dvp) {
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) states[(idx * KP + chained(m, 4 * qd + r)) * dvp + col] = S[m][r];
    }

    Frag<3> sf[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) sf[s] = split(S[2 * s], S[2 * s + 1]);
    // x = v - c (K S), o = e (Q S), per tile of sixteen tokens in chained order
    f32x4 o[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      f32x4 ks = {}, qs = {};
      const int row = chained(m, i) * TileK::kLd + 8 * qd;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        Frag<N> fk, fq;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          fk.t[n] = row_frag(&sk[n][row + 32 * s]);
          if constexpr (!STATES) fq.t[n] = row_frag(&sq[n][row + 32 * s]);
        }
        ks = mul(fk, sf[s], ks);
        if constexpr (!STATES) qs = mul<NO>(fq, sf[s], qs);
      }
      const int tok = chained(m, 4 * qd);
      x[m] -= *reinterpret_cast<const f32x4*>(&svec[tok]) * ks;
      o[m] = *reinterpret_cast<const f32x4*>(&svec[2 * kC + tok]) * qs;
    }
    // u = (T diag(beta)) x
    const Frag<3> xf[2] = {split(x[0], x[1]), split(x[2], x[3])};
    f32x4 u[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      u[m] = f32x4{};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (lower_frag(m, s) < 0) continue;
        Frag<3> ft;
#pragma unroll
        for (int n = 0; n < 3; ++n)
          ft.t[n] = *reinterpret_cast<const bf16x8*>(st + ((lower_frag(m, s) * 3 + n) * 64 + lane) * 16);
        u[m] = mul(ft, xf[s], u[m]);
      }
    }
    // o += P u
    if constexpr (!STATES) {
      const Frag<3> uf[2] = {split(u[0], u[1]), split(u[2], u[3])};
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (lower_frag(m, s) < 0) continue;
          Frag<NO> fp;
#pragma unroll
          for (int n = 0; n < NO; ++n)
            fp.t[n] = *reinterpret_cast<const bf16x8*>(sp + ((lower_frag(m, s) * NO + n) * 64 + lane) * 16);
          o[m] = mul<NO>(fp, uf[s], o[m]);
        }
      const Buffer rows = rows_of(op + t0 * out_t, L - t0 < kC ? L - t0 : kC, out_t, a.dv);
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          store1(rows, live_col ? o_lane + (32 * (m >> 1) + 4 * (m & 1) + r) * o_row : kOutside, IO(o[m][r]));
    } else if (col < dvp) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) values[(idx * kC + chained(m, 4 * qd + r)) * dvp + col] = u[m][r];
    }
    // S = last S + K^T (d u)
#pragma unroll
    for (int m = 0; m < 4; ++m) u[m] *= *reinterpret_cast<const f32x4*>(&svec[kC + chained(m, 4 * qd)]);
    const Frag<3> df[2] = {split(u[0], u[1]), split(u[2], u[3])};
    const float last = svec[3 * kC];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      S[m] *= last;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<N> fk;
#pragma unroll
        for (int n = 0; n < N; ++n) fk.t[n] = col_frag(sk[n], TileK::kLd, 32 * s + 8 * qd, chained(m, 4 * (i & 3)));
        S[m] = mul(fk, df[s], S[m]);
      }
    }
  }
  if constexpr (STATES) return;
  // tokens past the row's length: zeros (those of its last chunk were written above)
  if (live_col)
    for (int t = live_chunks * kC + qd; t < L; t += 4) op[t * out_t + col] = IO(0.0f);
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int dim = chained(m, 4 * qd + r);
      if (dim < a.dk && live_col) a.h_last[(bh * a.dk + dim) * a.dv + col] = S[m][r];
    }
}

}  // namespace delta
}  // namespace sscan
