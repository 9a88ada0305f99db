// sscan_delta.hip -- forward kernels of the gated delta rule: the chunk-local factors
// (prep), the walk over chunks, and the token-by-token kernel for decode and for
// sequences of a few tokens.
#include "sscan_delta.h"

#include "sscan_delta_chunk.h"
#include "sscan_delta_device.h"
#include "sscan_delta_prep.h"

namespace sscan {
namespace delta {

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

template <typename IO, int KP, int W>
hipError_t launch_walk(const DeltaArgs& a, const DeltaPlan& p, char* ws, hipStream_t stream) {
  const int wide = wide_flags<IO>(a), nvb = (a.dv + 16 * W - 1) / (16 * W), n = int(p.nchunk);
  char *ft = ws + p.off_t, *fp = ws + p.off_p;
  float* vec = reinterpret_cast<float*>(ws + p.off_vec);
  const int64_t bh = a.batch * a.hv;
  delta_prep_kernel<IO, KP, false>
      <<<dim3(unsigned(bh * n)), 256, 0, stream>>>(a, n, ft, fp, nullptr, vec, wide);
  const WalkArgs w{n, nvb, p.nseg, p.seg_chunks, p.dvp, wide, ft, fp, vec, nullptr, nullptr,
                   reinterpret_cast<float*>(ws + p.off_ends), reinterpret_cast<float*>(ws + p.off_moves)};
  if (p.nseg > 1) {
    constexpr int kIdent = (KP + 16 * W - 1) / (16 * W);
    delta_chunk_kernel<IO, KP, W, kEnds>
        <<<dim3(unsigned(bh * p.nseg * (nvb + kIdent))), 64 * W, 0, stream>>>(a, w, kVecFloats);
  }
  if (p.nseg > 2)
    delta_carry_kernel<KP, 4, false>
        <<<dim3(unsigned(bh * ((p.dvp + 63) / 64))), 256, 0, stream>>>(w.moves, w.ends, p.nseg, p.dvp, (p.dvp + 63) / 64);
  delta_chunk_kernel<IO, KP, W, kOut><<<dim3(unsigned(bh * p.nseg * nvb)), 64 * W, 0, stream>>>(a, w, kVecFloats);
  return hipGetLastError();
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
  if (p.kp == 64)
    return p.waves == 8 ? launch_walk<IO, 64, 8>(a, p, ws, stream) : launch_walk<IO, 64, 4>(a, p, ws, stream);
  return p.waves == 8 ? launch_walk<IO, 128, 8>(a, p, ws, stream) : launch_walk<IO, 128, 4>(a, p, ws, stream);
}

}  // namespace delta

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Segments a row is walked in.  One CU holds one block of a walk, so a walk takes
// ceil(blocks / CUs) times its chunks; in units of the time of one chunk of the output
// walk, a chunk of the transitions' walk takes 3/4 and a step of the chain between
// segments 1/2.
static int choose_segments(int64_t heads, int64_t nchunk, int nvb, int nkb) {
  constexpr int64_t kCus = 256;
  const auto rounds = [](int64_t blocks) { return double((blocks + kCus - 1) / kCus); };
  int best = 1;
  double least = rounds(heads * nvb) * double(nchunk);
  for (int n = 2; n <= 64 && nchunk / n >= 4; ++n) {
    const double chunks = double((nchunk + n - 1) / n);
    const double cost = rounds(heads * nvb * n) * chunks +
                        0.75 * rounds(heads * (nvb * (n - 1) + nkb * (n - 2))) * chunks + 0.5 * (n - 2) + 2.0;
    if (cost < 0.9 * least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

DeltaPlan make_delta_plan(int64_t batch, int64_t len, int hk, int hv, int dk, int dv, bool io_bf16) {
  (void)hk;
  DeltaPlan p{};
  p.nchunk = (len + kDeltaChunk - 1) / kDeltaChunk;
  p.recurrent = len <= kDeltaRecurrentMax;
  p.kp = dk <= 64 ? 64 : 128;
  p.dvp = (dv + 31) / 32 * 32;
  p.waves = dv > 64 ? 8 : 4;
  if (p.recurrent) return p;
  const int cols = 16 * p.waves;
  const int64_t heads = batch * hv;
  p.nseg = choose_segments(heads, p.nchunk, (dv + cols - 1) / cols, (p.kp + cols - 1) / cols);
  p.seg_chunks = int((p.nchunk + p.nseg - 1) / p.nseg);
  p.nseg = int((p.nchunk + p.seg_chunks - 1) / p.seg_chunks);
  const size_t n = size_t(heads) * size_t(p.nchunk);
  p.off_t = 0;
  p.off_p = p.off_t + round256(n * delta::kFrags * 3 * delta::kFragBytes);
  p.off_vec = p.off_p + round256(n * delta::kFrags * (io_bf16 ? 2 : 3) * delta::kFragBytes);
  p.off_ends = p.off_vec + round256(n * delta::kVecFloats * 4);
  const size_t segs = p.nseg > 1 ? size_t(heads) * size_t(p.nseg) * size_t(p.kp) * 4 : 0;
  p.off_moves = p.off_ends + round256(segs * size_t(p.dvp));
  p.workspace_bytes = p.off_moves + round256(segs * size_t(p.kp));
  return p;
}

hipError_t launch_delta_fwd(const DeltaArgs& a, const DeltaPlan& p, char* workspace, hipStream_t stream) {
  return a.io_bf16 ? delta::launch_fwd<delta::bf16>(a, p, workspace, stream)
                   : delta::launch_fwd<float>(a, p, workspace, stream);
}

}  // namespace sscan
