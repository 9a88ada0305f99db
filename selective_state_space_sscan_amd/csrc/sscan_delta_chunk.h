// sscan_delta_chunk.h -- the gated delta rule's walk over chunks, shared by the forward
// pass and by the recomputation of the states in the backward pass.
#pragma once

#include "sscan_delta.h"
#include "sscan_delta_device.h"

namespace sscan {
namespace delta {

// A wave owns sixteen columns of S for the whole sequence (KP x 16, in the accumulator
// layout) and walks the chunks in order; columns are independent, so waves never
// exchange data: every product's result is the next product's B factor in the same
// lane.  A block is four waves (64 columns) that share the chunk's K, Q, V tiles and
// the fragments of T and P through LDS.
// STATES: the backward pass's recomputation, which leaves every chunk's entry state
// [KP][dvp] and U [64][dvp] in float32 instead of the output and the last state.
template <typename IO, int KP, bool STATES>
__global__ __launch_bounds__(256) void delta_chunk_kernel(DeltaArgs a, int nchunk, int nvb, const char* frag_t,
                                                          const char* frag_p, const float* vec, float* states,
                                                          float* values, int dvp, int wide) {
  constexpr int N = Io<IO>::kN, NO = Io<IO>::kOutTerms;
  constexpr int kTiles = KP / 16, kSteps = KP / 32, kVecs = STATES ? kVecFloatsBwd : kVecFloats;
  constexpr int kLdV = std::is_same<IO, bf16>::value ? 72 : 68;
  typedef Tile<KP> TileK;
  __shared__ __attribute__((aligned(16))) bf16 sk[N][TileK::kElems];
  __shared__ __attribute__((aligned(16))) bf16 sq[STATES ? 1 : N][STATES ? 8 : TileK::kElems];
  __shared__ __attribute__((aligned(16))) IO sv[kC * kLdV];
  __shared__ __attribute__((aligned(16))) char st[kFrags * 3 * kFragBytes];
  __shared__ __attribute__((aligned(16))) char sp[STATES ? 16 : kFrags * NO * kFragBytes];
  __shared__ __attribute__((aligned(16))) float svec[kVecFloats];

  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6, i = lane & 15, qd = lane >> 4;
  const int64_t blk = blockIdx.x;
  const int64_t bh = blk / nvb;
  const int64_t b = bh / a.hv;
  const int h = int(bh % a.hv), hq = h / (a.hv / a.hk);
  const int col_blk = int(blk % nvb) * 64, col = col_blk + 16 * wave + i;
  const int L = int(a.len), Lb = row_len(a.lengths, b, a.len);
  const int live_chunks = (Lb + kC - 1) / kC;
  const IO* kp = static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h;
  const IO* qp = static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h;
  const IO* vp = static_cast<const IO*>(a.v) + b * a.sv.b + h * a.sv.h;
  IO* op = static_cast<IO*>(a.out) + (b * a.len * a.hv + h) * a.dv;
  const int64_t out_t = int64_t(a.hv) * a.dv;
  const bool wide_qk = wide & 1, wide_v = wide & 2, wide_o = wide & 4;

  f32x4 S[kTiles];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int dim = chained(m, 4 * qd + r);
      S[m][r] = (a.h0 && dim < a.dk && col < a.dv) ? a.h0[(bh * a.dk + dim) * a.dv + col] : 0.0f;
    }

  for (int c = 0; c < nchunk; ++c) {
    const int t0 = c * kC;
    if (STATES && c >= live_chunks) break;
    if (c < live_chunks) {
      const int64_t idx = bh * nchunk + c;
      if (STATES && col < dvp) {
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) states[(idx * KP + chained(m, 4 * qd + r)) * dvp + col] = S[m][r];
      }
      __syncthreads();  // the last chunk's readers of the tiles are done
      for (int u = tid; u < kC * KP / 8; u += 256) {
        const int row = u / (KP / 8), d8 = (u % (KP / 8)) * 8;
        const bool in = t0 + row < Lb;
        const auto fk = as_frag(load8(kp + (t0 + row) * a.sk.t + d8, in ? a.dk - d8 : 0, wide_qk));
#pragma unroll
        for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x8*>(&sk[n][row * TileK::kLd + d8]) = fk.t[n];
        if constexpr (!STATES) {
          const auto fq = as_frag(load8(qp + (t0 + row) * a.sq.t + d8, in ? a.dk - d8 : 0, wide_qk));
#pragma unroll
          for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x8*>(&sq[n][row * TileK::kLd + d8]) = fq.t[n];
        }
      }
      for (int u = tid; u < kC * 8; u += 256) {
        const int row = u / 8, c8 = (u % 8) * 8;
        const bool in = t0 + row < Lb;
        const auto x = load8(vp + (t0 + row) * a.sv.t + col_blk + c8, in ? a.dv - col_blk - c8 : 0, wide_v);
        *reinterpret_cast<typename Io<IO>::V8*>(&sv[row * kLdV + c8]) = x;
      }
      for (int u = tid; u < kFrags * 3 * 64; u += 256)
        reinterpret_cast<u32x4*>(st)[u] = reinterpret_cast<const u32x4*>(frag_t + idx * kFrags * 3 * kFragBytes)[u];
      if constexpr (!STATES)
        for (int u = tid; u < kFrags * NO * 64; u += 256)
          reinterpret_cast<u32x4*>(sp)[u] = reinterpret_cast<const u32x4*>(frag_p + idx * kFrags * NO * kFragBytes)[u];
      if (tid < kVecFloats) svec[tid] = vec[idx * kVecs + tid];
      __syncthreads();

      Frag<3> sf[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) sf[s] = split(S[2 * s], S[2 * s + 1]);
      // x = v - c (K S), o = e (Q S), per tile of sixteen tokens in chained order
      f32x4 x[4], o[4];
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
        const f32x4 vc = *reinterpret_cast<const f32x4*>(&svec[tok]);
        const f32x4 ve = *reinterpret_cast<const f32x4*>(&svec[2 * kC + tok]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[m][r] = to_f32(sv[(tok + r) * kLdV + 16 * wave + i]) - vc[r] * ks[r];
          o[m][r] = ve[r] * qs[r];
        }
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
      if constexpr (STATES) continue;
      // the output takes the place of this wave's columns of V
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) sv[(chained(m, 4 * qd) + r) * kLdV + 16 * wave + i] = IO(o[m][r]);
    }
    __syncthreads();
    for (int u = tid; u < kC * 8; u += 256) {
      const int row = u / 8, c8 = (u % 8) * 8, t = t0 + row;
      if (t >= L) continue;
      IO* dst = op + t * out_t + col_blk + c8;
      const int left = a.dv - col_blk - c8;
      typename Io<IO>::V8 y = {};
      if (c < live_chunks) y = *reinterpret_cast<const typename Io<IO>::V8*>(&sv[row * kLdV + c8]);
      if (wide_o) {
        if (left > 0) *reinterpret_cast<typename Io<IO>::V8*>(dst) = y;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) dst[j] = y[j];
      }
    }
  }
  if constexpr (STATES) return;
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int dim = chained(m, 4 * qd + r);
      if (dim < a.dk && col < a.dv) a.h_last[(bh * a.dk + dim) * a.dv + col] = S[m][r];
    }
}

}  // namespace delta
}  // namespace sscan
