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

__device__ __forceinline__ f32x8 read8(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

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
  // column i of the block's inverse; a row's coefficients are the same in every lane,
  // and a value is subtracted from all later rows as soon as it is known
  float t[16];
  f32x4 row[16][4];
#pragma unroll
  for (int r = 1; r < 16; ++r)
#pragma unroll
    for (int k = 0; k < r; k += 4) row[r][k / 4] = *reinterpret_cast<const f32x4*>(&M[(d0 + r) * kLdM + d0 + k]);
#pragma unroll
  for (int r = 0; r < 16; ++r) t[r] = r == i ? 1.0f : 0.0f;
#pragma unroll
  for (int k = 0; k < 15; ++k)
#pragma unroll
    for (int r = k + 1; r < 16; ++r) t[r] -= row[r][k / 4][k % 4] * t[k];
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
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k < J) continue;
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

// x of another lane by a DPP control; 0 where the control names none.
template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t w = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(w), kCtrl, kRows, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(w >> 32), kCtrl, kRows, 0xf, false);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// Inclusive sum over the wave's 64 lanes in double: decays are exponentials of
// differences of these sums, which float32 sums of large negative g would lose.
__device__ __forceinline__ double wave_running_sum(double x) {
  x += dpp<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8
  x += dpp<0x112, 0xf>(x);
  x += dpp<0x114, 0xf>(x);
  x += dpp<0x118, 0xf>(x);
  x += dpp<0x142, 0xa>(x);  // lane 15 of the row before, into rows 1 and 3
  x += dpp<0x143, 0xc>(x);  // lane 31, into rows 2 and 3
  return x;
}

__device__ __forceinline__ double lane_of(double x, int lane) {
  const uint64_t w = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(int(w), lane), hi = __builtin_amdgcn_readlane(int(w >> 32), lane);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// One block per (batch row, value head, chunk).  Wave w computes rows 16 w .. + 15 of
// K K^T and Q K^T against the tokens up to them.  The decay of a pair in one tile of
// sixteen is its own exponential; of a pair in two tiles the product of two, through the
// last token of the earlier tile, both at most 1 (for g <= 0) and never smaller than the
// product: seven exponentials a lane instead of thirty-two.  BWD: T, T^T and P^T.
//
// Bound by the latency of the inversion's chain (fifteen dependent steps, then three rounds
// of block products in float32), hidden only by the other blocks of a CU: 8192 chunks and
// heads (32768 tokens of 16 heads of 128) 170 us, 2048 of them 42 us, 54 with BWD's
// transposes; what the 8192 read and write, 0.4 GB, would take 85 us.
template <typename IO, int KP, bool BWD>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, int nchunk, char* frag_t, char* frag_p,
                                                         char* frag_tt, float* vec, int wide) {
  constexpr int N = Io<IO>::kN, kSteps = KP / 32;
  __shared__ __attribute__((aligned(16))) float pmat[kC * kLdM];
  __shared__ __attribute__((aligned(16))) float tmat[kC * kLdM];
  __shared__ double gsum[kC];
  __shared__ __attribute__((aligned(16))) float sbeta[kC];
  __shared__ float srk[kC], srq[kC], from[3][kC], to_end[kC];

  const int tid = int(threadIdx.x), lane = tid & 63, wave = wave_id(), i = lane & 15, qd = lane >> 4;
  // fewer than 2^24 blocks: 32-bit divisions
  const unsigned bh = blockIdx.x / unsigned(nchunk), row_b = bh / unsigned(a.hv);
  const int c = int(blockIdx.x - bh * unsigned(nchunk)), h = int(bh - row_b * unsigned(a.hv));
  const int hq = int(unsigned(h) / (unsigned(a.hv) / unsigned(a.hk)));
  const int64_t idx = blockIdx.x, b = row_b;
  const int Lb = row_len(a.lengths, b, a.len), t0 = c * kC;
  if (t0 >= Lb) return;
  const bool wide_qk = wide & 1;
  const int rows = Lb - t0 < kC ? Lb - t0 : kC;
  const Buffer kb = rows_of(static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h + t0 * a.sk.t, rows, a.sk.t, a.dk);
  const Buffer qb = rows_of(static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h + t0 * a.sq.t, rows, a.sq.t, a.dk);

  typename Io<IO>::V8 xk[kSteps], xq[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int d8 = 32 * s + 8 * qd, row = 16 * wave + i;
    const int left = row < rows ? a.dk - d8 : 0;
    load8<IO>(kb, (row * int(a.sk.t) + d8) * int(sizeof(IO)), left, wide_qk, &xk[s]);
    load8<IO>(qb, (row * int(a.sq.t) + d8) * int(sizeof(IO)), left, wide_qk, &xq[s]);
  }
  // every wave has all tokens' running sums of g, and computes one of the tables
  const int t = t0 + lane;
  float g = 0.0f, beta = 0.0f;
  if (t < Lb) {
    g = clamp_decay(a.g[b * a.sg.b + t * a.sg.t + h * a.sg.h]);
    beta = a.beta[b * a.sb.b + t * a.sb.t + h * a.sb.h];
  }
  const double sum = wave_running_sum(double(g));
  if (wave < 3) {
    const double ref = lane_of(sum, 16 * wave + 15);
    from[wave][lane] = lane > 16 * wave + 15 ? expf(float(sum - ref)) : 0.0f;
  } else {
    const double ref = lane < 16 ? lane_of(sum, 15) : lane < 32 ? lane_of(sum, 31) : lane < 48 ? lane_of(sum, 47)
                                                                                              : lane_of(sum, 63);
    to_end[lane] = expf(float(ref - sum));
    gsum[lane] = sum;
    sbeta[lane] = beta;
  }

  f32x4 kk[4], qk[4];
  {
    Frag<N> fk[kSteps], fq[kSteps];
    float ssq = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      fk[s] = as_frag(xk[s]);
      fq[s] = as_frag(xq[s]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ssq += to_f32(xq[s][j]) * to_f32(xq[s][j]);
    }
    ssq += __shfl_xor(ssq, 16);
    ssq += __shfl_xor(ssq, 32);
    // the keys' squares are the diagonal of K K^T: lane (qd, i) with i / 4 == qd holds key i's
    float diag = 0.0f;
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      kk[ct] = qk[ct] = f32x4{};
      if (ct > wave) continue;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        Frag<N> fb = fk[s];
        if (ct != wave) {
          const int d8 = 32 * s + 8 * qd;
          typename Io<IO>::V8 x;
          load8<IO>(kb, ((16 * ct + i) * int(a.sk.t) + d8) * int(sizeof(IO)), 16 * ct + i < rows ? a.dk - d8 : 0, wide_qk, &x);
          fb = as_frag(x);
        }
        kk[ct] = mul(fk[s], fb, kk[ct]);
        qk[ct] = mul(fq[s], fb, qk[ct]);
      }
      if (ct == wave) {
#pragma unroll
        for (int r = 0; r < 4; ++r) diag = (i & 3) == r ? kk[ct][r] : diag;
      }
    }
    float rq = 1.0f, rk = 1.0f;
    if (a.qk_norm) {
      rq = 1.0f / sqrtf(ssq + 1e-6f);
      rk = 1.0f / sqrtf(diag + 1e-6f);
    }
    if ((i >> 2) == qd) {
      srq[16 * wave + i] = rq;
      srk[16 * wave + i] = rk;
    }
  }
  __syncthreads();
  if (wave == 0) {
    const float into = expf(float(sum)), rest = expf(float(lane_of(sum, 63) - sum));
    float* v = vec + idx * (BWD ? kVecFloatsBwd : kVecFloats);
    v[lane] = into * srk[lane];
    v[kC + lane] = rest * srk[lane];
    v[2 * kC + lane] = a.scale * into * srq[lane];
    v[3 * kC + lane] = expf(float(lane_of(sum, 63)));
    if constexpr (BWD) {
      v[4 * kC + lane] = beta;
      v[5 * kC + lane] = srk[lane];
      v[6 * kC + lane] = srq[lane];
    }
  }
  {
    const int row = 16 * wave + 4 * qd;
    float fk[4], fq[4];  // beta rk, scale rq of this lane's four rows
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      fk[r] = sbeta[row + r] * srk[row + r];
      fq[r] = a.scale * srq[row + r];
    }
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      if (ct > (wave | 1)) continue;  // only the tile that shares a fragment with the diagonal is read beyond it
      const int tj = 16 * ct + i;
      const float rk = srk[tj], end = to_end[tj];
      const double sum_j = gsum[tj];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float decay = 0.0f;
        if (ct < wave) decay = from[ct < 3 ? ct : 0][row + r] * end;
        if (ct == wave) decay = expf(float(gsum[row + r] - sum_j));
        decay *= rk;
        const float t = fk[r] * decay * kk[ct][r], p = fq[r] * decay * qk[ct][r];
        tmat[(row + r) * kLdM + tj] = ct < wave || tj < row + r ? t : 0.0f;
        pmat[(row + r) * kLdM + tj] = ct < wave || tj <= row + r ? p : 0.0f;
      }
    }
  }
  __syncthreads();
  invert_unit_lower(tmat, wave);

  constexpr int kKinds = BWD ? 3 : 2;
#pragma unroll
  for (int n = 0; n < (kKinds * kFrags + 3) / 4; ++n) {
    const int task = wave + 4 * n;
    if (task >= kKinds * kFrags) break;
    const int kind = task / kFrags, f = task % kFrags;  // 0: T, 1: P (BWD: P^T), 2: T^T
    const bool upper = BWD && kind > 0;
    const int m = upper ? upper_m(f) : lower_m(f), s = upper ? upper_s(f) : lower_s(f);
    const int row = chained(m, i), k0 = 32 * s + 8 * qd;
    const float* from_mat = kind == 1 ? pmat : tmat;
    f32x8 x;
    if (upper) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = from_mat[(k0 + j) * kLdM + row];
    } else {
      x = read8(&from_mat[row * kLdM + k0]);
    }
    if (kind == 0) x *= read8(&sbeta[k0]);
    const Frag<3> fr = split(x);
    char* dst = (kind == 0 ? frag_t : kind == 1 ? frag_p : frag_tt) + (idx * kFrags + f) * kTerms * kFragBytes;
#pragma unroll
    for (int k = 0; k < kTerms; ++k) *reinterpret_cast<bf16x8*>(dst + (k * 64 + lane) * 16) = fr.t[k];
  }
}

// Which loads may be 16 bytes wide (per-call, from alignment and sizes): bit 0 q and
// k, bit 1 v, bit 2 out, bit 3 the states.  All of them single, rows of 2-byte alignment:
// 4 x 2048 tokens of 8 heads 225 us against 123, a document of 32768 of 16 heads 1495
// against 722, gradients of 4 x 2048 509 against 371.
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
