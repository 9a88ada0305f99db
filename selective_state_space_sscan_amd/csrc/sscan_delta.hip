// sscan_delta.hip -- forward kernels of the gated delta rule: the chunk-local factors
// (prep), the walk over chunks, and the token-by-token kernel for decode and for
// sequences of a few tokens.
#include "sscan_delta.h"

#include "sscan_delta_device.h"
#include "sscan_delta_prep.h"

namespace sscan {
namespace delta {

// ---- the walk over chunks -----------------------------------------------------------
//
// A wave owns sixteen columns of S for the whole sequence (KP x 16, in the accumulator
// layout) and walks the chunks in order; columns are independent, so waves never
// exchange data: every product's result is the next product's B factor in the same
// lane.  A block is four waves (64 columns) that share the chunk's K, Q, V tiles and
// the fragments of T and P through LDS.
template <typename IO, int KP>
__global__ __launch_bounds__(256) void delta_chunk_kernel(DeltaArgs a, int nchunk, int nvb, const char* frag_t,
                                                          const char* frag_p, const float* vec, int wide) {
  constexpr int N = Io<IO>::kN, NO = Io<IO>::kOutTerms;
  constexpr int kTiles = KP / 16, kSteps = KP / 32;
  constexpr int kLdV = std::is_same<IO, bf16>::value ? 72 : 68;
  typedef Tile<KP> TileK;
  __shared__ __attribute__((aligned(16))) bf16 sk[N][TileK::kElems];
  __shared__ __attribute__((aligned(16))) bf16 sq[N][TileK::kElems];
  __shared__ __attribute__((aligned(16))) IO sv[kC * kLdV];
  __shared__ __attribute__((aligned(16))) char st[kFrags * 3 * kFragBytes];
  __shared__ __attribute__((aligned(16))) char sp[kFrags * NO * kFragBytes];
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
    if (c < live_chunks) {
      const int64_t idx = bh * nchunk + c;
      __syncthreads();  // the last chunk's readers of the tiles are done
      for (int u = tid; u < kC * KP / 8; u += 256) {
        const int row = u / (KP / 8), d8 = (u % (KP / 8)) * 8;
        const bool in = t0 + row < Lb;
        const auto fk = as_frag(load8(kp + (t0 + row) * a.sk.t + d8, in ? a.dk - d8 : 0, wide_qk));
        const auto fq = as_frag(load8(qp + (t0 + row) * a.sq.t + d8, in ? a.dk - d8 : 0, wide_qk));
#pragma unroll
        for (int n = 0; n < N; ++n) {
          *reinterpret_cast<bf16x8*>(&sk[n][row * TileK::kLd + d8]) = fk.t[n];
          *reinterpret_cast<bf16x8*>(&sq[n][row * TileK::kLd + d8]) = fq.t[n];
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
      for (int u = tid; u < kFrags * NO * 64; u += 256)
        reinterpret_cast<u32x4*>(sp)[u] = reinterpret_cast<const u32x4*>(frag_p + idx * kFrags * NO * kFragBytes)[u];
      if (tid < kVecFloats) svec[tid] = vec[idx * kVecFloats + tid];
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
            fq.t[n] = row_frag(&sq[n][row + 32 * s]);
          }
          ks = mul(fk, sf[s], ks);
          qs = mul<NO>(fq, sf[s], qs);
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
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int dim = chained(m, 4 * qd + r);
      if (dim < a.dk && col < a.dv) a.h_last[(bh * a.dk + dim) * a.dv + col] = S[m][r];
    }
}

// ---- token by token -----------------------------------------------------------------
//
// A wave owns 32 columns of S: lane (rg, cg) holds rows rg NR .. + NR - 1 of columns
// 4 cg .. + 3.  One pass over S gives S'^T k and S'^T q together (o = S'^T q + (k.q) u),
// so a decode step reads and writes the state once.
template <typename IO, int NR>
__global__ __launch_bounds__(256) void delta_recurrent_kernel(DeltaArgs a, int ncol, int64_t waves, int wide) {
  const int lane = lane_id(), rg = lane >> 3, cg = lane & 7;
  const int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (w >= waves) return;
  const int64_t bh = w / ncol, b = bh / a.hv;
  const int h = int(bh % a.hv), hq = h / (a.hv / a.hk);
  const int col = int(w % ncol) * 32 + 4 * cg, row0 = rg * NR;
  const int L = int(a.len), Lb = row_len(a.lengths, b, a.len);
  const bool wide_qk = wide & 1, wide_s = wide & 8;
  const IO* kp = static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h + row0;
  const IO* qp = static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h + row0;
  const IO* vp = static_cast<const IO*>(a.v) + b * a.sv.b + h * a.sv.h + col;
  const float* gp = a.g + b * a.sg.b + h * a.sg.h;
  const float* bp = a.beta + b * a.sb.b + h * a.sb.h;
  IO* op = static_cast<IO*>(a.out) + (b * a.len * a.hv + h) * a.dv + col;
  const int64_t out_t = int64_t(a.hv) * a.dv;
  const int64_t state = (bh * a.dk + row0) * a.dv + col;
  const int cols = a.dv - col, rows = a.dk - row0;

  f32x4 S[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    S[r] = f32x4{};
    if (a.h0 && r < rows) {
      const float* p = a.h0 + state + int64_t(r) * a.dv;
      if (wide_s) {
        if (cols > 0) S[r] = *reinterpret_cast<const f32x4*>(p);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < cols) S[r][j] = p[j];
      }
    }
  }
  for (int t = 0; t < Lb; ++t) {
    float k[NR], q[NR];
#pragma unroll
    for (int r8 = 0; r8 < NR; r8 += 8) {
      const auto k8 = load8(kp + t * a.sk.t + r8, rows - r8, wide_qk);
      const auto q8 = load8(qp + t * a.sq.t + r8, rows - r8, wide_qk);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        k[r8 + j] = to_f32(k8[j]);
        q[r8 + j] = to_f32(q8[j]);
      }
    }
    f32x4 v = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < cols) v[j] = to_f32(vp[t * a.sv.t + j]);
    const float decay = expf(clamp_decay(gp[t * a.sg.t])), beta = bp[t * a.sb.t];
    f32x4 ks = {}, qs = {};
    float kk = 0, qq = 0, kq = 0;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      ks += k[r] * S[r];
      qs += q[r] * S[r];
      kk += k[r] * k[r];
      qq += q[r] * q[r];
      kq += k[r] * q[r];
    }
#pragma unroll
    for (int m = 8; m < 64; m *= 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ks[j] += __shfl_xor(ks[j], m);
        qs[j] += __shfl_xor(qs[j], m);
      }
      kk += __shfl_xor(kk, m);
      qq += __shfl_xor(qq, m);
      kq += __shfl_xor(kq, m);
    }
    const float rk = a.qk_norm ? 1.0f / sqrtf(kk + 1e-6f) : 1.0f, rq = a.qk_norm ? 1.0f / sqrtf(qq + 1e-6f) : 1.0f;
    const f32x4 u = beta * (v - (decay * rk) * ks), ku = rk * u;
    const f32x4 o = (a.scale * rq) * (decay * qs + kq * ku);
#pragma unroll
    for (int r = 0; r < NR; ++r) S[r] = decay * S[r] + k[r] * ku;
    if (rg == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cols) op[t * out_t + j] = IO(o[j]);
    }
  }
  if (rg == 0)
    for (int t = Lb; t < L; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cols) op[t * out_t + j] = IO(0.0f);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (r >= rows) continue;
    float* p = a.h_last + state + int64_t(r) * a.dv;
    if (wide_s) {
      if (cols > 0) *reinterpret_cast<f32x4*>(p) = S[r];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < cols) p[j] = S[r][j];
    }
  }
}

template <typename IO>
hipError_t launch_fwd(const DeltaArgs& a, const DeltaPlan& p, char* ws, hipStream_t stream) {
  const int wide = wide_flags<IO>(a);
  if (p.recurrent) {
    const int ncol = (a.dv + 31) / 32;
    const int64_t waves = a.batch * a.hv * ncol;
    const dim3 grid{unsigned((waves + 3) / 4)};
    if (a.dk <= 64)
      delta_recurrent_kernel<IO, 8><<<grid, 256, 0, stream>>>(a, ncol, waves, wide);
    else
      delta_recurrent_kernel<IO, 16><<<grid, 256, 0, stream>>>(a, ncol, waves, wide);
    return hipGetLastError();
  }
  const int nvb = (a.dv + 63) / 64, n = int(p.nchunk);
  char *ft = ws + p.off_t, *fp = ws + p.off_p;
  float* vec = reinterpret_cast<float*>(ws + p.off_vec);
  const dim3 prep{unsigned(a.batch * a.hk * n)}, grid{unsigned(a.batch * a.hv * nvb)};
  if (a.dk <= 64) {
    delta_prep_kernel<IO, 64, false><<<prep, 256, 0, stream>>>(a, n, ft, fp, nullptr, vec, wide);
    delta_chunk_kernel<IO, 64><<<grid, 256, 0, stream>>>(a, n, nvb, ft, fp, vec, wide);
  } else {
    delta_prep_kernel<IO, 128, false><<<prep, 256, 0, stream>>>(a, n, ft, fp, nullptr, vec, wide);
    delta_chunk_kernel<IO, 128><<<grid, 256, 0, stream>>>(a, n, nvb, ft, fp, vec, wide);
  }
  return hipGetLastError();
}

}  // namespace delta

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

DeltaPlan make_delta_plan(int64_t batch, int64_t len, int hk, int hv, int dk, int dv, bool io_bf16) {
  (void)hk;
  (void)dk;
  (void)dv;
  DeltaPlan p{};
  p.nchunk = (len + kDeltaChunk - 1) / kDeltaChunk;
  p.recurrent = len <= kDeltaRecurrentMax;
  if (p.recurrent) return p;
  const size_t n = size_t(batch) * size_t(hv) * size_t(p.nchunk);
  p.off_t = 0;
  p.off_p = p.off_t + round256(n * delta::kFrags * 3 * delta::kFragBytes);
  p.off_vec = p.off_p + round256(n * delta::kFrags * (io_bf16 ? 2 : 3) * delta::kFragBytes);
  p.workspace_bytes = p.off_vec + round256(n * delta::kVecFloats * 4);
  return p;
}

hipError_t launch_delta_fwd(const DeltaArgs& a, const DeltaPlan& p, char* workspace, hipStream_t stream) {
  return a.io_bf16 ? delta::launch_fwd<delta::bf16>(a, p, workspace, stream)
                   : delta::launch_fwd<float>(a, p, workspace, stream);
}

}  // namespace sscan
