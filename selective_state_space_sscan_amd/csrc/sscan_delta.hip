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
// so a decode step reads and writes the state once and is bound by that traffic (128
// sequences of 32 heads of 128 x 128: 537 MB).  WIDE: 16-byte accesses to the state, whose
// rows allow it for dv a multiple of four; QK to q and k, where their size, strides and
// alignment allow it.  Otherwise every element is loaded by itself (q and k: one row of 16
// heads 4.1 us a token against 3.7, of 8 tokens 15.3 against 12.2; the state: 128 sequences
// 145 against 86).

// Sum over the eight row groups (lane bits 3 to 5), in every lane.
__device__ __forceinline__ float group_rows_sum(float x) {
  x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x128, 0xf, 0xf, true));
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = __builtin_bit_cast(float, unsigned(p[0])) + __builtin_bit_cast(float, unsigned(p[1]));
  const unsigned v = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return __builtin_bit_cast(float, unsigned(r[0])) + __builtin_bit_cast(float, unsigned(r[1]));
}

template <typename IO, int NR, bool WIDE, bool QK>
__global__ __launch_bounds__(256) void delta_recurrent_kernel(DeltaArgs a, unsigned ncol, unsigned waves) {
  const int lane = lane_id(), rg = lane >> 3, cg = lane & 7;
  const unsigned w = __builtin_amdgcn_readfirstlane(blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6));
  if (w >= waves) return;
  const unsigned bh = w / ncol, row_b = bh / unsigned(a.hv);
  const int64_t b = row_b;
  const int h = int(bh - row_b * unsigned(a.hv)), hq = int(unsigned(h) / (unsigned(a.hv) / unsigned(a.hk)));
  const int col = int(w - bh * ncol) * 32 + 4 * cg, row0 = rg * NR;
  const int L = int(a.len), Lb = row_len(a.lengths, b, a.len);
  const IO* kp = static_cast<const IO*>(a.k) + b * a.sk.b + hq * a.sk.h;
  const IO* qp = static_cast<const IO*>(a.q) + b * a.sq.b + hq * a.sq.h;
  const IO* vp = static_cast<const IO*>(a.v) + b * a.sv.b + h * a.sv.h;
  const float* gp = a.g + b * a.sg.b + h * a.sg.h;
  const float* bp = a.beta + b * a.sb.b + h * a.sb.h;
  const int64_t out_t = int64_t(a.hv) * a.dv;
  IO* op = static_cast<IO*>(a.out) + (b * a.len * a.hv + h) * a.dv;
  const uint32_t state_bytes = uint32_t(a.dk * a.dv * 4);
  // a lane's columns in a state row (kOutside: none)
  const int at = col < a.dv ? (row0 * a.dv + col) * 4 : kOutside;

  const auto state_io = [&](const float* p, auto body) {
    const Buffer s = buffer_of(p + int64_t(bh) * a.dk * a.dv, state_bytes);
#pragma unroll
    for (int r = 0; r < NR; ++r) body(s, at + r * a.dv * 4, r);
  };
  f32x4 S[NR];
  if (a.h0) {
    state_io(a.h0, [&](Buffer s, int off, int r) {
      if constexpr (WIDE) {
        S[r] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(s, off, 0, 0));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x;
          load1(s, col + j < a.dv ? off + 4 * j : kOutside, &x);
          S[r][j] = x;
        }
      }
    });
  } else {
#pragma unroll
    for (int r = 0; r < NR; ++r) S[r] = f32x4{};
  }
  for (int t = 0; t < Lb; ++t) {
    const Buffer kb = buffer_of(kp + t * a.sk.t, uint32_t(a.dk * sizeof(IO)));
    const Buffer qb = buffer_of(qp + t * a.sq.t, uint32_t(a.dk * sizeof(IO)));
    const Buffer vb = buffer_of(vp + t * a.sv.t, uint32_t(a.dv * sizeof(IO)));
    typename Io<IO>::V8 k8[NR / 8], q8[NR / 8];
#pragma unroll
    for (int n = 0; n < NR / 8; ++n) {
      load8<IO>(kb, (row0 + 8 * n) * int(sizeof(IO)), a.dk - row0 - 8 * n, QK, &k8[n]);
      load8<IO>(qb, (row0 + 8 * n) * int(sizeof(IO)), a.dk - row0 - 8 * n, QK, &q8[n]);
    }
    IO v4[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) load1(vb, (col + j) * int(sizeof(IO)), &v4[j]);
    const float decay = expf(clamp_decay(gp[t * a.sg.t])), beta = bp[t * a.sb.t];
    float k[NR], q[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      k[r] = to_f32(k8[r / 8][r % 8]);
      q[r] = to_f32(q8[r / 8][r % 8]);
    }
    f32x4 ks = {}, qs = {}, v;
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
    for (int j = 0; j < 4; ++j) {
      ks[j] = group_rows_sum(ks[j]);
      qs[j] = group_rows_sum(qs[j]);
      v[j] = to_f32(v4[j]);
    }
    kk = group_rows_sum(kk);
    qq = group_rows_sum(qq);
    kq = group_rows_sum(kq);
    const float rk = a.qk_norm ? 1.0f / sqrtf(kk + 1e-6f) : 1.0f, rq = a.qk_norm ? 1.0f / sqrtf(qq + 1e-6f) : 1.0f;
    const f32x4 u = beta * (v - (decay * rk) * ks), ku = rk * u;
    const f32x4 o = (a.scale * rq) * (decay * qs + kq * ku);
#pragma unroll
    for (int r = 0; r < NR; ++r) S[r] = decay * S[r] + k[r] * ku;
    if (rg == 0) {
      const Buffer ob = buffer_of(op + t * out_t, uint32_t(a.dv * sizeof(IO)));
#pragma unroll
      for (int j = 0; j < 4; ++j) store1(ob, (col + j) * int(sizeof(IO)), IO(o[j]));
    }
  }
  if (rg == 0)
    for (int t = Lb; t < L; ++t) {
      const Buffer ob = buffer_of(op + t * out_t, uint32_t(a.dv * sizeof(IO)));
#pragma unroll
      for (int j = 0; j < 4; ++j) store1(ob, (col + j) * int(sizeof(IO)), IO(0.0f));
    }
  state_io(a.h_last, [&](Buffer s, int off, int r) {
    if constexpr (WIDE) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[r]), s, off, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) store1(s, col + j < a.dv ? off + 4 * j : kOutside, S[r][j]);
    }
  });
}

template <typename IO, int NR>
hipError_t launch_recurrent(const DeltaArgs& a, hipStream_t stream) {
  const int wide = wide_flags<IO>(a), ncol = (a.dv + 31) / 32;
  const unsigned waves = unsigned(a.batch * a.hv * ncol);
  // Blocks of one wave while there are at most two a CU: a small batch then uses as many CUs
  // as it has waves.  One token of 16 heads of 128 x 128, one wave a block and four (us):
  // 64 waves 3.7 and 4.3, 512 waves 5.2 and 5.6, 1024 waves 7.1 and 7.0, 2048 10.5 and 10.1.
  const unsigned per_block = waves <= 512 ? 1 : 4, blocks = (waves + per_block - 1) / per_block;
  const auto run = [&](auto states, auto qk) {
    delta_recurrent_kernel<IO, NR, decltype(states)::value, decltype(qk)::value>
        <<<dim3(blocks), 64 * per_block, 0, stream>>>(a, unsigned(ncol), waves);
  };
  if ((wide & 9) == 9)
    run(std::true_type(), std::true_type());
  else if (wide & 8)
    run(std::true_type(), std::false_type());
  else
    run(std::false_type(), std::false_type());
  return hipGetLastError();
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
    delta_carry_kernel<KP, false>
        <<<dim3(unsigned(bh * (p.dvp / 16))), 2 * KP, 0, stream>>>(w.moves, w.ends, p.nseg, p.dvp);
  delta_chunk_kernel<IO, KP, W, kOut><<<dim3(unsigned(bh * p.nseg * nvb)), 64 * W, 0, stream>>>(a, w, kVecFloats);
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_fwd(const DeltaArgs& a, const DeltaPlan& p, char* ws, hipStream_t stream) {
  if (p.recurrent) return a.dk <= 64 ? launch_recurrent<IO, 8>(a, stream) : launch_recurrent<IO, 16>(a, stream);
  if constexpr (std::is_same<IO, bf16>::value)  // float32 walks have four waves
    if (p.waves == 8) return p.kp == 64 ? launch_walk<IO, 64, 8>(a, p, ws, stream) : launch_walk<IO, 128, 8>(a, p, ws, stream);
  return p.kp == 64 ? launch_walk<IO, 64, 4>(a, p, ws, stream) : launch_walk<IO, 128, 4>(a, p, ws, stream);
}

}  // namespace delta

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Segments a row is walked in, by a model of the walks' times in units of one chunk of
// one output walk alone on its CU (4.5 us at 128 x 128 by four waves, 5.6 by eight): a CU
// holds one block (so it does of the output walks and of eight waves; of the transitions and
// states of four waves with keys of 64 it holds two, and the model counts their rounds twice);
// chunks take up to 1.4 times as long when every CU is busy; a walk has 2 units of its own
// for its first loads; a chunk of the transitions' walk takes 3/4, and its blocks end at
// different times, so its rounds count fractionally; a step of the chain between segments
// takes 1 (1/4 for keys of 64).  Measured against forced counts, all of them bf16, 128 x 128
// (us a call): 64 heads of 32 chunks 175 in 4 segments (the model's choice), 167 in 3, 207 in
// 8, 223 whole; 16 heads of 512 chunks 706 in 16 (its choice), 823 in 8, 781 in 12, 755 in
// 32, 3200 whole; 256 heads of 16 chunks 200 whole (its choice), 331 in 2.
static int choose_segments(int64_t heads, int64_t nchunk, int nvb, int nkb, int kp) {
  const auto walk = [](int64_t blocks, double rounds, double chunks) {
    const double busy = blocks < 256 ? double(blocks) / 256.0 : 1.0;
    return rounds * chunks * (1.0 + 0.4 * busy) + 2.0;
  };
  const auto output = [&](int n) {
    const int64_t blocks = heads * nvb * n;
    return walk(blocks, double((blocks + 255) / 256), double((nchunk + n - 1) / n));
  };
  int best = 1;
  double least = 0.97 * output(1);
  for (int n = 2; n <= 64 && nchunk / n >= 2; ++n) {
    const double chunks = double((nchunk + n - 1) / n);
    const int64_t blocks = heads * (int64_t(nvb) * (n - 1) + int64_t(nkb) * (n - 2));
    const double rounds = blocks < 256 ? 1.0 : double(blocks) / 256.0;
    const double cost = output(n) + walk(blocks, rounds, 0.75 * chunks) + (n - 2) * (kp == 64 ? 0.25 : 1.0) + 1.0;
    if (cost < least) {
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
  // Waves of a walk's block.  Eight share a chunk's tiles between 128 columns, four take a
  // CU for themselves and end a chunk sooner (4.5 us against 5.6): four for float32 (whose
  // registers eight waves spill: 2 x 2048 tokens of 8 heads 125 us against 136, one row of
  // 500 72 against 108) and where there are few chunks for the GPU (bf16, 4 heads of 500
  // tokens 50 us against 60; 64 heads of 2048 195 against 181; 256 heads of 1024 248 against
  // 212).
  p.waves = dv > 64 && io_bf16 && batch * hv * p.nchunk >= 1024 ? 8 : 4;
  if (p.recurrent) return p;
  const int cols = 16 * p.waves;
  const int64_t heads = batch * hv;
  p.nseg = choose_segments(heads, p.nchunk, (dv + cols - 1) / cols, (p.kp + cols - 1) / cols, p.kp);
  p.seg_chunks = int((p.nchunk + p.nseg - 1) / p.nseg);
  p.nseg = int((p.nchunk + p.seg_chunks - 1) / p.seg_chunks);
  const size_t n = size_t(heads) * size_t(p.nchunk);
  p.off_t = 0;
  p.off_p = p.off_t + round256(n * delta::kFrags * 3 * delta::kFragBytes);
  p.off_vec = p.off_p + round256(n * delta::kFrags * 3 * delta::kFragBytes);
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
