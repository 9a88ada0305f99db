// sscan_delta_prep.h -- chunk-local factors of the gated delta rule, shared by its
// forward and backward passes: T diag(beta) = (I + A)^-1 diag(beta), the masked and
// decayed P = scale (Q K^T . D) (backward: T^T and P^T too), and the per-token factors,
// laid out as the matrix instruction's A fragments.
#pragma once

#include "sscan_delta.h"
#include "sscan_delta_device.h"

namespace sscan {
namespace delta {

constexpr int kLdM = 68;  // floats between rows of a 64 x 64 LDS matrix

// c + M[r0.., c0..] b for 16 x 16 blocks in float32, b in the result layout.
__device__ __forceinline__ f32x4 block_mul(const float* M, int r0, int c0, f32x4 b, f32x4 c) {
  const int i = lane_id() & 15, qd = lane_id() >> 4;
  const f32x4 x = *reinterpret_cast<const f32x4*>(&M[(r0 + i) * kLdM + c0 + 4 * qd]);
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], b[r], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ f32x4 block_read(const float* M, int r0, int c0) {
  const int i = lane_id() & 15, qd = lane_id() >> 4;
  f32x4 b;
#pragma unroll
  for (int r = 0; r < 4; ++r) b[r] = M[(r0 + 4 * qd + r) * kLdM + c0 + i];
  return b;
}

__device__ __forceinline__ void block_write(float* M, int r0, int c0, f32x4 b) {
  const int i = lane_id() & 15, qd = lane_id() >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) M[(r0 + 4 * qd + r) * kLdM + c0 + i] = b[r];
}

// M (strictly lower triangular A, zeros elsewhere) becomes (I + A)^-1, by four waves:
// the diagonal blocks of 16 by forward substitution (which stays accurate however
// strongly the keys are correlated), the others from
// T_ij = -T_ii (sum_{j <= k < i} A_ik T_kj), 32-row halves last.
__device__ __forceinline__ void invert_unit_lower(float* M, int wave) {
  const int i = lane_id() & 15, qd = lane_id() >> 4, d0 = 16 * wave;
  float t[16];  // column i of the block's inverse
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float x = r == i ? 1.0f : 0.0f;
#pragma unroll
    for (int k = 0; k < r; ++k) x -= M[(d0 + r) * kLdM + d0 + k] * t[k];
    t[r] = x;
  }
  // all of this wave's reads of its block come before its writes (one wave, in order)
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if ((r >> 2) == qd) M[(d0 + r) * kLdM + d0 + i] = t[r];
  __syncthreads();
  if (wave < 2) {
    const int r0 = 32 * wave + 16, c0 = 32 * wave;
    const f32x4 y = block_mul(M, r0, c0, block_read(M, c0, c0), f32x4{});
    block_write(M, r0, c0, -block_mul(M, r0, r0, y, f32x4{}));
  }
  __syncthreads();
  const int I = 2 + (wave >> 1), J = wave & 1;
  f32x4 y2 = {}, y3 = {};
  for (int k = J; k < 2; ++k) {
    const f32x4 t_kj = block_read(M, 16 * k, 16 * J);
    y2 = block_mul(M, 32, 16 * k, t_kj, y2);
    if (I == 3) y3 = block_mul(M, 48, 16 * k, t_kj, y3);
  }
  f32x4 z = block_mul(M, 16 * I, 32, y2, f32x4{});
  if (I == 3) z = block_mul(M, 48, 48, y3, z);
  __syncthreads();  // A's blocks are read by two waves each
  block_write(M, 16 * I, 16 * J, -z);
  __syncthreads();
}

// Inclusive sum over the wave's 64 lanes in double: decays are exponentials of
// differences of these sums, which float32 sums of large negative g would lose.
__device__ __forceinline__ double wave_running_sum(double x) {
  const int lane = lane_id();
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const double y = __shfl_up(x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// One block per (batch row, key head, chunk); the value heads that share the key head
// reuse its K K^T and Q K^T.  BWD: the transposed fragments as well, three terms each.
template <typename IO, int KP, bool BWD>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, int nchunk, char* frag_t, char* frag_p,
                                                         char* frag_tt, float* vec, int wide) {
  constexpr int N = Io<IO>::kN, NP = BWD ? 3 : Io<IO>::kOutTerms, kSteps = KP / 32;
  __shared__ __attribute__((aligned(16))) float kk[kC * kLdM];
  __shared__ __attribute__((aligned(16))) float qk[kC * kLdM];
  __shared__ __attribute__((aligned(16))) float mat[kC * kLdM];
  __shared__ double gsum[kC];
  __shared__ float sbeta[kC], srk[kC], srq[kC];

  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6, i = lane & 15, qd = lane >> 4;
  const int c = int(blockIdx.x % unsigned(nchunk));
  const int64_t bhk = blockIdx.x / unsigned(nchunk);
  const int64_t b = bhk / a.hk;
  const int hq = int(bhk % a.hk), share = a.hv / a.hk;
  const int Lb = row_len(a.lengths, b, a.len), t0 = c * kC;
  if (t0 >= Lb) return;
  const bool wide_qk = wide & 1;
  const IO* kp = static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h;
  const IO* qp = static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h;

  // K K^T and Q K^T: wave w takes tokens 16 w .. 16 w + 15 against all earlier ones
  {
    const int tok = t0 + 16 * wave + i;
    const bool in = tok < Lb;
    Frag<N> fk[kSteps], fq[kSteps];
    float ssq = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d8 = 32 * s + 8 * qd;
      fk[s] = as_frag(load8(kp + tok * a.sk.t + d8, in ? a.dk - d8 : 0, wide_qk));
      const auto q8 = load8(qp + tok * a.sq.t + d8, in ? a.dk - d8 : 0, wide_qk);
      fq[s] = as_frag(q8);
#pragma unroll
      for (int j = 0; j < 8; ++j) ssq += to_f32(q8[j]) * to_f32(q8[j]);
    }
    ssq += __shfl_xor(ssq, 16);
    ssq += __shfl_xor(ssq, 32);
    if (qd == 0) srq[16 * wave + i] = a.qk_norm ? 1.0f / sqrtf(ssq + 1e-6f) : 1.0f;
    for (int ct = 0; ct <= wave; ++ct) {
      const int tc = t0 + 16 * ct + i;
      f32x4 xk = {}, xq = {};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d8 = 32 * s + 8 * qd;
        const auto fb = as_frag(load8(kp + tc * a.sk.t + d8, tc < Lb ? a.dk - d8 : 0, wide_qk));
        xk = mul(fk[s], fb, xk);
        xq = mul(fq[s], fb, xq);
      }
      block_write(kk, 16 * wave, 16 * ct, xk);
      block_write(qk, 16 * wave, 16 * ct, xq);
    }
  }
  __syncthreads();
  if (tid < kC) srk[tid] = a.qk_norm ? 1.0f / sqrtf(kk[tid * kLdM + tid] + 1e-6f) : 1.0f;

  for (int hh = 0; hh < share; ++hh) {
    const int h = hq * share + hh;
    const int64_t idx = (b * a.hv + h) * nchunk + c;
    __syncthreads();
    if (wave == 0) {
      const int t = t0 + lane;
      float g = 0.0f, beta = 0.0f;
      if (t < Lb) {
        g = clamp_decay(a.g[b * a.sg.b + t * a.sg.t + h * a.sg.h]);
        beta = a.beta[b * a.sb.b + t * a.sb.t + h * a.sb.h];
      }
      const double sum = wave_running_sum(double(g)), end = __shfl(sum, 63);
      gsum[lane] = sum;
      sbeta[lane] = beta;
      const float into = expf(float(sum)), rest = expf(float(end - sum));
      float* v = vec + idx * (BWD ? kVecFloatsBwd : kVecFloats);
      v[lane] = into * srk[lane];
      v[kC + lane] = rest * srk[lane];
      v[2 * kC + lane] = a.scale * into * srq[lane];
      v[3 * kC + lane] = expf(float(end));
      if constexpr (BWD) {
        v[4 * kC + lane] = beta;
        v[5 * kC + lane] = srk[lane];
        v[6 * kC + lane] = srq[lane];
      }
    }
    __syncthreads();
    for (int e = tid; e < kC * kC; e += 256) {
      const int r = e / kC, j = e % kC;
      float x = 0.0f;
      if (j < r) x = sbeta[r] * expf(float(gsum[r] - gsum[j])) * srk[r] * srk[j] * kk[r * kLdM + j];
      mat[r * kLdM + j] = x;
    }
    __syncthreads();
    invert_unit_lower(mat, wave);

    constexpr int kKinds = BWD ? 3 : 2;
    for (int task = wave; task < kKinds * kFrags; task += 4) {
      const int kind = task / kFrags, f = task % kFrags;  // 0: T, 1: P (BWD: P^T), 2: T^T
      const bool upper = BWD && kind > 0;
      const int m = upper ? (f < 4 ? f >> 1 : f - 2) : (f < 2 ? f : (f + 2) >> 1);
      const int s = upper ? (f < 4 ? f & 1 : 1) : (f < 2 ? 0 : f & 1);
      const int row = chained(m, i), k0 = 32 * s + 8 * qd;
      f32x8 x;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = upper ? k0 + j : row, q = upper ? row : k0 + j;  // matrix row (later token), column
        if (kind == 1)
          x[j] = q <= r ? a.scale * srq[r] * srk[q] * expf(float(gsum[r] - gsum[q])) * qk[r * kLdM + q] : 0.0f;
        else
          x[j] = kind == 0 ? mat[r * kLdM + q] * sbeta[q] : mat[r * kLdM + q];
      }
      const Frag<3> fr = split(x);
      const int terms = kind == 1 ? NP : 3;
      char* dst = (kind == 0 ? frag_t : kind == 1 ? frag_p : frag_tt) + (idx * kFrags + f) * terms * kFragBytes;
#pragma unroll
      for (int n = 0; n < 3; ++n)
        if (n < terms) *reinterpret_cast<bf16x8*>(dst + (n * 64 + lane) * 16) = fr.t[n];
    }
  }
}

// Which loads may be 16 bytes wide (per-call, from alignment and sizes): bit 0 q and
// k, bit 1 v, bit 2 out, bit 3 the states.
template <typename IO>
int wide_flags(const DeltaArgs& a) {
  const auto ok = [](const void* p, const DeltaStride& s) {
    const int64_t n = 16 / int64_t(sizeof(IO));
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s.b % n == 0 && s.t % n == 0 && s.h % n == 0;
  };
  int w = 0;
  if (a.dk % 8 == 0 && ok(a.q, a.sq) && ok(a.k, a.sk)) w |= 1;
  if (a.dv % 8 == 0 && ok(a.v, a.sv)) w |= 2;
  if (a.dv % 8 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0) w |= 4;
  if (a.dv % 4 == 0) w |= 8;
  return w;
}

}  // namespace delta
}  // namespace sscan
