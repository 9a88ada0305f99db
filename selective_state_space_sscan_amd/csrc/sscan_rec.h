// sscan_rec.h -- launch interface between the C ABI (sscan_rec_capi.cpp) and the gfx950
// kernels of the gated recurrence (sscan_rec.hip, sscan_rec_bwd.hip), of activations in 8
// bits (sscan_pack8.hip) and of the layer norm (sscan_layer_norm.hip).  Not part of the
// public ABI.
//
// Per batch row and channel, with a float32 state h:
//   a_t = exp(-c softplus(lam) r_t), r_t = sigmoid(g_t), w_t = sqrt(1 - a_t^2),
//   or a_t = exp(g_t), w_t = 1;
//   h_t = a_t h_{t-1} + w_t s_t x_t, s_t = sigmoid(i_t);   out_t = h_t silu(z_t)
// The gradients, with D_t the adjoint of h_t (D after the last token: dh_last):
//   D_t = dout_t silu(z_t) + a_{t+1} D_{t+1},  dz_t = dout_t h_t silu'(z_t),
//   dx_t = D_t w_t s_t,  di_t = D_t w_t x_t s_t (1 - s_t),
//   dlog a_t = D_t (a_t h_{t-1} - s_t x_t a_t^2 / w_t)        (the second term with lam),
//   dg_t = dlog a_t, or -dlog a_t c softplus(lam) r_t (1 - r_t) and
//   dlam = -sum_t dlog a_t c r_t sigmoid(lam)
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace sscan {

constexpr int kPackBlock = 64;       // elements that share a scale

struct RecIn {
  const void* p;                     // [batch, len, dim] by these strides, dim contiguous
  int64_t b, t;                      // elements between batch rows and tokens
};

struct RecKept {
  int8_t *x, *g, *i, *z;             // [batch, len, dim]
  float *xs, *gs, *is, *zs;          // [batch, len, ceil(dim / 64)]
};

struct RecArgs {
  RecIn x, g, i, z;                  // i.p, z.p nullable
  const float* lam;                  // nullable, [dim]
  const int32_t* lengths;            // nullable, [batch]
  const float* h0;                   // nullable, [batch, dim]
  float* h_last;                     // [batch, dim] (may equal h0)
  void* out;                         // [batch, len, dim] contiguous
  RecKept kept;                      // forward: written, where x is not NULL
  int64_t batch, len, dim;
  float c;
  int reverse, io_bf16;
};

struct RecBwdArgs {
  RecArgs f;                         // the forward's inputs; read from f.kept where kept.x is not NULL
  const void* dout;                  // contiguous
  const float* dh_last;              // nullable
  void *dx, *dg, *di, *dz;
  float *dlam, *dh0;                 // nullable
};

size_t rec_workspace(int64_t batch, int64_t len, int64_t dim, bool io_bf16);
size_t rec_bwd_workspace(int64_t batch, int64_t len, int64_t dim, bool io_bf16);
hipError_t launch_rec_fwd(const RecArgs& a, char* workspace, hipStream_t stream);
hipError_t launch_rec_step(const RecArgs& a, hipStream_t stream);
hipError_t launch_rec_bwd(const RecBwdArgs& a, char* workspace, hipStream_t stream);

struct PackArgs {
  const void* x;                     // [rows, size], rows x_stride apart
  int64_t x_stride;
  int8_t* q;                         // [rows, size]
  float* scale;                      // [rows, ceil(size / 64)]
  void* out;                         // unpack: contiguous
  int64_t rows, size;
  int io_bf16;
};

hipError_t launch_pack8(const PackArgs& a, hipStream_t stream);
hipError_t launch_unpack8(const PackArgs& a, hipStream_t stream);

struct LayerNormArgs {
  const void* x;                     // forward: [rows, size] io dtype; backward: the total, residual dtype
  int64_t x_stride;
  const void* residual;              // forward, nullable
  const float *weight, *bias;        // nullable, [size]
  void *out, *total;                 // forward; total nullable
  const void *dout, *dtotal;         // backward; dtotal nullable
  void *dx, *dresidual;              // backward; dresidual nullable
  float *dweight, *dbias;            // backward, nullable
  int64_t rows, size;
  float eps;
  int io_bf16, res_bf16;
};

size_t layer_norm_bwd_workspace(int64_t rows, int64_t size);
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t stream);
hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, float* workspace, hipStream_t stream);

// out[k][e] = sum over the nblocks rows of partial[row][k][e], k < parts <= 3, in order
// (out[k] NULL: not wanted); rows of `parts * size` floats.
hipError_t launch_row_sums(const float* partial, float* const* out, int parts, int64_t size, int64_t nblocks,
                           hipStream_t stream);

}  // namespace sscan
