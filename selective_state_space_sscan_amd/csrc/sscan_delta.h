// sscan_delta.h -- launch interface between the C ABI (sscan_delta_capi.cpp) and the
// gfx950 kernels of the gated delta rule (sscan_delta.hip, sscan_delta_bwd.hip).
// Not part of the public ABI.
//
// Per batch row and value head, with a state S [dk, dv] held in float32:
//   S' = exp(g_t) S,  u_t = beta_t (v_t - S'^T k_t),  S <- S' + k_t u_t^T,
//   o_t = scale S^T q_t
// In chunks of C = 64 tokens, with G_i the running sum of g inside the chunk, S0 the
// state entering it and D_ij = exp(G_i - G_j) for i >= j:
//   A_ij = beta_i D_ij (k_i . k_j)  (i > j),   T = (I + A)^-1
//   U    = T diag(beta) (V - diag(exp G) K S0)
//   O    = scale (diag(exp G) Q S0 + (Q K^T . D) U)
//   S1   = exp(G_C) S0 + K^T diag(exp(G_C - G_j)) U
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace sscan {

constexpr int kDeltaChunk = 64;
constexpr int kDeltaMaxK = 128;      // key size (a state's rows, held in registers)
constexpr int kDeltaMaxV = 256;      // value size
constexpr int64_t kDeltaMaxStride = 1 << 23;  // elements between tokens: a chunk's rows stay within 2^31 bytes
// Sequences of at most this many tokens take the token-by-token kernel, whose time grows
// with them.  At heads of 128 x 128, by tokens and by chunks (us a call): one row of 8 heads,
// bf16, 13.5 and 18.9 for 8 tokens, 18.1 and 18.9 for 12, 23 and 19 for 16; 8 rows of 16 heads
// 15.3 and 21.5, 20.0 and 21.1, 25 and 21; 128 rows of 16 heads 63 and 114, 81 and 109, 106
// and 108; float32 gains up to 16 and more (22 and 23, 24 and 27, 103 and 210).
constexpr int kDeltaRecurrentMax = 10;

struct DeltaStride {
  int64_t b, t, h;                   // elements between batch rows, tokens and heads
};

struct DeltaArgs {
  const void *q, *k, *v;             // [batch, len, heads, size] io dtype by these strides, size contiguous
  const float *g, *beta;             // [batch, len, v_heads] by these strides
  DeltaStride sq, sk, sv, sg, sb;
  const int32_t* lengths;            // nullable, [batch]: tokens of each row (clamped to 0..len)
  const float* h0;                   // nullable, [batch, v_heads, dk, dv]
  float* h_last;                     // [batch, v_heads, dk, dv] (may equal h0)
  void* out;                         // [batch, len, v_heads, dv] io dtype, contiguous
  int64_t batch, len;
  int hk, hv, dk, dv;
  float scale;
  int qk_norm, io_bf16;
};

struct DeltaBwdArgs {
  DeltaArgs f;                       // the forward's inputs (out and h_last unused)
  const void* dout;                  // [batch, len, v_heads, dv] io dtype, contiguous
  const float* dh_last;              // nullable
  void *dq, *dk, *dv;                // contiguous, io dtype
  float *dg, *dbeta;                 // [batch, len, v_heads]
  float* dh0;                        // nullable, [batch, v_heads, dk, dv]
};

// Workspace (byte offsets, 256-aligned).
struct DeltaPlan {
  int64_t nchunk;                    // chunks per row
  int recurrent;                     // token-by-token kernel, no workspace
  int kp;                            // dk rounded up to 64 or 128
  int dvp;                           // dv rounded up to 32
  int waves;                         // waves (sixteen value columns each) of a walk's block
  int nseg, seg_chunks;              // segments of a row walked at once, chunks in each
  size_t off_t, off_p, off_vec;      // forward: fragments of T and of the masked Q K^T; per-token factors
  size_t off_ends, off_moves;        // segments' end (entry) states and transitions
  size_t workspace_bytes;
};

// Backward: the transposed fragments as well, the corrected values U and the adjoint X~
// in float32, the state and its adjoint at every chunk's edge, and the adjoints between
// segments.
struct DeltaBwdPlan {
  DeltaPlan f;
  size_t off_tt, off_pt, off_u, off_y, off_s, off_ds, off_back;
  size_t workspace_bytes;
};

DeltaPlan make_delta_plan(int64_t batch, int64_t len, int hk, int hv, int dk, int dv, bool io_bf16);
DeltaBwdPlan make_delta_bwd_plan(int64_t batch, int64_t len, int hk, int hv, int dk, int dv, bool io_bf16);
hipError_t launch_delta_fwd(const DeltaArgs& a, const DeltaPlan& p, char* workspace, hipStream_t stream);
hipError_t launch_delta_bwd(const DeltaBwdArgs& a, const DeltaBwdPlan& p, char* workspace, hipStream_t stream);

// RMS norms fused with what stands beside them in a block.
constexpr int kNormMaxSize = 8192;   // eight elements for each of 1024 threads
constexpr int64_t kNormMaxHeads = 1 << 20;  // with a weight each

struct GatedNormArgs {
  const void *x, *z;                 // [rows, heads, size] io dtype by these strides, size contiguous
  int64_t xr, xh, zr, zh;            // elements between rows and heads
  const float* weight;               // nullable, [size] or [heads, size]
  int per_head;
  const void* dout;                  // backward: contiguous
  void* out;                         // forward
  void *dx, *dz;                     // backward, contiguous
  float* dweight;                    // backward, nullable
  int64_t rows, heads, size;
  float eps;
  int gate_first, io_bf16;
};

struct AddNormArgs {
  const void* x;                     // [rows, size] io dtype, contiguous
  const void* residual;              // forward: nullable; backward: the sum the forward stored
  const float *weight, *scale, *post_weight;  // nullable, [size]
  void *out, *residual_out;          // forward
  const void *dout, *dresidual_out;  // backward; dresidual_out nullable
  void *dx, *dresidual;              // backward
  float *dweight, *dscale, *dpost_weight;  // backward, nullable
  int64_t rows, size;
  float eps;
  int io_bf16, res_bf16;
};

size_t gated_norm_bwd_workspace(int64_t rows, int64_t heads, int64_t size);
size_t add_norm_bwd_workspace(int64_t rows, int64_t size);
hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream);
hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, float* workspace, hipStream_t stream);
hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream);
hipError_t launch_add_norm_bwd(const AddNormArgs& a, float* workspace, hipStream_t stream);

}  // namespace sscan
