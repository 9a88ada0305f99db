// sscan_rec_capi.cpp -- C ABI of the gated recurrence, of activations in 8 bits and of the
// layer norm: argument checks, then one call into the kernel launchers.  Every check comes
// before any HIP call, so the validate entry points work without a GPU.
#include "sscan.h"

#include <cmath>
#include <cstdint>

#include "sscan_check.h"
#include "sscan_delta.h"
#include "sscan_rec.h"

namespace {

using namespace sscan::check;

constexpr int64_t kMaxStride = int64_t(1) << 26;  // elements between tokens: a tile's sixteen stay within 2^32 bytes
constexpr int64_t kMaxLen = int64_t(1) << 30, kMaxDim = int64_t(1) << 24, kMaxTiles = int64_t(1) << 22;

int64_t blocks_of(int64_t size) { return (size + sscan::kPackBlock - 1) / sscan::kPackBlock; }

struct RecView {
  sscan::RecArgs a;
  size_t esz, bytes, state_bytes, lam_bytes, kept_bytes, scale_bytes;  // of contiguous tensors
  Range in[4], lam, lengths, h0, kept[8];
  bool no_rows, no_tokens;
};

// The ranges of the inputs kept in 8 bits, where they are given: x and g always, i and z
// by `i` and `z` (forward: as the call has them; backward: as given).
int view_kept(const sscan_rec_kept* k, bool i, bool z, RecView* w) {
  if (!k) return SSCAN_OK;
  int8_t* const q[4] = {k->x, k->g, k->i, k->z};
  float* const s[4] = {k->x_scale, k->g_scale, k->i_scale, k->z_scale};
  const bool want[4] = {true, true, i, z};
  for (int n = 0; n < 4; ++n) {
    if (!want[n]) {
      if (q[n] || s[n]) return SSCAN_ERR_UNSUPPORTED;
      continue;
    }
    if (!w->no_rows && !w->no_tokens && (!q[n] || !s[n])) return SSCAN_ERR_NULL;
    if (!aligned(s[n], 4)) return SSCAN_ERR_ALIGN;
    w->kept[2 * n] = range_of(q[n], w->kept_bytes);
    w->kept[2 * n + 1] = range_of(s[n], w->scale_bytes);
  }
  w->a.kept = sscan::RecKept{k->x, k->g, k->i, k->z, k->x_scale, k->g_scale, k->i_scale, k->z_scale};
  return SSCAN_OK;
}

// Sizes, codes, pointers and strides of the inputs, and the ranges they cover.  `kept`: the
// inputs come in 8 bits, p has none.
int view_rec(const sscan_rec_params* p, bool kept, RecView* w) {
  if (!p) return SSCAN_ERR_NULL;
  if (p->batch < 0 || p->len < 0 || p->dim < 0) return SSCAN_ERR_SHAPE;
  if (!dtype_ok(p->io_dtype) || (p->reverse != 0 && p->reverse != 1) || !std::isfinite(p->c) || p->c < 0)
    return SSCAN_ERR_UNSUPPORTED;
  w->no_rows = p->batch == 0 || p->dim == 0;
  w->no_tokens = p->len == 0;
  w->esz = dtype_size(p->io_dtype);
  if (p->len > kMaxLen || p->dim > kMaxDim) return SSCAN_ERR_SHAPE;
  const int64_t n = product({p->batch, p->len, p->dim}), ns = product({p->batch, p->dim}),
                tiles = product({p->batch, (p->dim + 63) / 64, p->len / 64 + 1});
  if (n < 0 || ns < 0 || tiles < 0 || tiles >= kMaxTiles) return SSCAN_ERR_SHAPE;
  w->bytes = size_t(n) * w->esz;
  w->state_bytes = size_t(ns) * 4;
  w->lam_bytes = size_t(p->dim) * 4;
  w->kept_bytes = size_t(n);
  w->scale_bytes = size_t(p->batch) * size_t(p->len) * size_t(blocks_of(p->dim)) * 4;
  const void* ptr[4] = {p->x, p->g, p->i, p->z};
  const int64_t* strides[4] = {p->x_stride, p->g_stride, p->i_stride, p->z_stride};
  if (kept && (p->x || p->g || p->i || p->z)) return SSCAN_ERR_UNSUPPORTED;
  if (!kept && !w->no_rows && !w->no_tokens && (!p->x || !p->g)) return SSCAN_ERR_NULL;
  if (!aligned(p->lam, 4) || !aligned(p->lengths, 4) || !aligned(p->h0, 4)) return SSCAN_ERR_ALIGN;
  sscan::RecIn in[4] = {};
  for (int k = 0; k < 4; ++k) {
    if (!ptr[k]) continue;
    if (!aligned(ptr[k], w->esz)) return SSCAN_ERR_ALIGN;
    const int64_t dims[2] = {p->batch, p->len}, e = extent(dims, strides[k], 2, p->dim);
    if (e < 0) return SSCAN_ERR_SHAPE;
    if (p->len > 1 && strides[k][1] >= kMaxStride) return SSCAN_ERR_UNSUPPORTED;  // a single token's is never used
    w->in[k] = range_of(ptr[k], w->no_rows || w->no_tokens ? 0 : size_t(e) * w->esz);
    in[k] = sscan::RecIn{ptr[k], strides[k][0], p->len > 1 ? strides[k][1] : 0};
  }
  w->lam = range_of(p->lam, w->lam_bytes);
  w->lengths = range_of(p->lengths, size_t(p->batch) * 4);
  w->h0 = range_of(p->h0, w->state_bytes);
  w->a = sscan::RecArgs{in[0], in[1], in[2], in[3], p->lam, p->lengths, p->h0, nullptr, nullptr, {}, p->batch, p->len,
                        p->dim, p->c, p->reverse, p->io_dtype == SSCAN_BF16};
  return SSCAN_OK;
}

bool clash_inputs(const Range& out, const RecView& w) {
  return clash(out, {w.in[0], w.in[1], w.in[2], w.in[3], w.lam, w.lengths});
}

int check_rec_fwd(const sscan_rec_params* p, const void* out, const float* h_last, const sscan_rec_kept* kept,
                  const void* workspace, size_t workspace_bytes, RecView* w) {
  int st = view_rec(p, false, w);
  if (st == SSCAN_OK) st = view_kept(kept, p->i != nullptr, p->z != nullptr, w);
  if (st != SSCAN_OK || w->no_rows) return st;
  if (!h_last || (!w->no_tokens && !out)) return SSCAN_ERR_NULL;
  if (!aligned(h_last, 4) || !aligned(out, w->esz)) return SSCAN_ERR_ALIGN;
  const size_t need = sscan::rec_workspace(p->batch, p->len, p->dim, w->a.io_bf16 != 0);
  st = check_workspace(workspace, workspace_bytes, need, 256);
  if (st != SSCAN_OK) return st;
  const Range o = range_of(out, w->bytes), s = range_of(h_last, w->state_bytes), ws = range_of(workspace, need);
  if (clash_inputs(o, *w) || clash(o, {w->h0, s, ws}) || clash_inputs(s, *w) || overlap(s, ws) ||
      (h_last != p->h0 && overlap(s, w->h0)) || clash_inputs(ws, *w) || overlap(ws, w->h0))
    return SSCAN_ERR_ALIAS;
  for (int i = 0; i < 8; ++i) {
    if (clash_inputs(w->kept[i], *w) || clash(w->kept[i], {w->h0, o, s, ws})) return SSCAN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(w->kept[i], w->kept[j])) return SSCAN_ERR_ALIAS;
  }
  return SSCAN_OK;
}

int check_rec_step(const sscan_rec_params* p, const float* state, const void* out, RecView* w) {
  if (!p) return SSCAN_ERR_NULL;
  if (p->len != 1) return SSCAN_ERR_SHAPE;
  if (p->h0 || p->reverse) return SSCAN_ERR_UNSUPPORTED;
  int st = view_rec(p, false, w);
  if (st != SSCAN_OK || w->no_rows) return st;
  if (!state || !out) return SSCAN_ERR_NULL;
  if (!aligned(state, 4) || !aligned(out, w->esz)) return SSCAN_ERR_ALIGN;
  const Range o = range_of(out, w->bytes), s = range_of(state, w->state_bytes);
  return clash_inputs(o, *w) || clash_inputs(s, *w) || overlap(o, s) ? SSCAN_ERR_ALIAS : SSCAN_OK;
}

int check_rec_bwd(const sscan_rec_params* p, const sscan_rec_kept* kept, const void* dout, const float* dh_last,
                  const sscan_rec_grads* grads, const void* workspace, size_t workspace_bytes, RecView* w) {
  if (!grads) return SSCAN_ERR_NULL;
  int st = view_rec(p, kept != nullptr, w);
  if (st == SSCAN_OK) st = view_kept(kept, kept && kept->i, kept && kept->z, w);
  if (st != SSCAN_OK) return st;
  const sscan_rec_grads& g = *grads;
  const bool i = kept ? kept->i != nullptr : p->i != nullptr, z = kept ? kept->z != nullptr : p->z != nullptr;
  if (g.dlam && !p->lam) return SSCAN_ERR_NULL;
  if (!w->no_rows && !w->no_tokens && (!dout || !g.dx || !g.dg || (i && !g.di) || (z && !g.dz))) return SSCAN_ERR_NULL;
  if ((g.di && !i) || (g.dz && !z)) return SSCAN_ERR_UNSUPPORTED;
  if (!aligned(dout, w->esz) || !aligned(g.dx, w->esz) || !aligned(g.dg, w->esz) || !aligned(g.di, w->esz) ||
      !aligned(g.dz, w->esz) || !aligned(g.dlam, 4) || !aligned(g.dh0, 4) || !aligned(dh_last, 4))
    return SSCAN_ERR_ALIGN;
  const size_t need = w->no_rows ? 0 : sscan::rec_bwd_workspace(p->batch, p->len, p->dim, w->a.io_bf16 != 0);
  st = check_workspace(workspace, workspace_bytes, need, 256);
  if (st != SSCAN_OK) return st;
  const Range outs[6] = {range_of(g.dx, w->bytes), range_of(g.dg, w->bytes),       range_of(g.di, w->bytes),
                         range_of(g.dz, w->bytes), range_of(g.dlam, w->lam_bytes), range_of(g.dh0, w->state_bytes)};
  const Range d = range_of(dout, w->bytes), dh = range_of(dh_last, w->state_bytes), ws = range_of(workspace, need);
  if (clash_inputs(ws, *w) || clash(ws, {w->h0, d, dh})) return SSCAN_ERR_ALIAS;
  for (int m = 0; m < 8; ++m)
    if (overlap(ws, w->kept[m])) return SSCAN_ERR_ALIAS;
  for (int n = 0; n < 6; ++n) {
    if (clash_inputs(outs[n], *w) || clash(outs[n], {w->h0, d, dh, ws})) return SSCAN_ERR_ALIAS;
    for (int m = 0; m < 8; ++m)
      if (overlap(outs[n], w->kept[m])) return SSCAN_ERR_ALIAS;
    for (int m = 0; m < n; ++m)
      if (overlap(outs[n], outs[m])) return SSCAN_ERR_ALIAS;
  }
  return SSCAN_OK;
}

// The sizes a workspace query is asked for, as the call itself checks them.
bool rec_sizes_ok(int64_t batch, int64_t len, int64_t dim, int io_dtype) {
  sscan_rec_params p{};
  p.batch = batch;
  p.len = len;
  p.dim = dim;
  p.io_dtype = io_dtype;
  RecView w{};
  const int st = view_rec(&p, true, &w);  // there are no pointers to check
  return st == SSCAN_OK && !w.no_rows;
}

// A tensor of rows in 8 bits: sizes, codes, pointers (x: io_dtype, strided; q, scale).
int check_pack8(const void* x, int64_t x_stride, int64_t rows, int64_t size, int io_dtype, const int8_t* q,
                const float* scale, bool reads_x, bool* empty) {
  if (rows < 0 || size < 0) return SSCAN_ERR_SHAPE;
  if (!dtype_ok(io_dtype)) return SSCAN_ERR_UNSUPPORTED;
  const int64_t n = product({rows, size}), e = extent(&rows, &x_stride, 1, size);
  if (n < 0 || e < 0) return SSCAN_ERR_SHAPE;
  *empty = n == 0;
  if (*empty) return SSCAN_OK;
  if (!x || !q || !scale) return SSCAN_ERR_NULL;
  if (!aligned(x, dtype_size(io_dtype)) || !aligned(scale, 4)) return SSCAN_ERR_ALIGN;
  const Range rx = range_of(x, size_t(e) * dtype_size(io_dtype)), rq = range_of(q, size_t(n)),
              rs = range_of(scale, size_t(rows) * size_t(blocks_of(size)) * 4);
  // packing writes q and scale, unpacking x
  if (overlap(rx, rq) || overlap(rx, rs) || (reads_x && overlap(rq, rs))) return SSCAN_ERR_ALIAS;
  return SSCAN_OK;
}

struct LayerView {
  sscan::LayerNormArgs a;
  size_t esz, rsz, bytes, res_bytes, vec_bytes;
  Range x, residual, weight, bias;
  bool empty;
};

int view_layer(const sscan_layer_norm_params* p, bool back, LayerView* w) {
  if (!p) return SSCAN_ERR_NULL;
  if (p->rows < 0) return SSCAN_ERR_SHAPE;
  if (p->size < 1 || p->size > sscan::kNormMaxSize || !dtype_ok(p->io_dtype) || !dtype_ok(p->residual_dtype) ||
      !std::isfinite(p->eps) || p->eps < 0)
    return SSCAN_ERR_UNSUPPORTED;
  w->empty = p->rows == 0;
  const int64_t n = product({p->rows, p->size}), e = extent(&p->rows, &p->x_stride, 1, p->size);
  if (n < 0 || e < 0) return SSCAN_ERR_SHAPE;
  w->esz = dtype_size(p->io_dtype);
  w->rsz = dtype_size(p->residual_dtype);
  const size_t xsz = back ? w->rsz : w->esz;
  w->bytes = size_t(n) * w->esz;
  w->res_bytes = size_t(n) * w->rsz;
  w->vec_bytes = size_t(p->size) * 4;
  if (!w->empty && !p->x) return SSCAN_ERR_NULL;
  if (!aligned(p->x, xsz) || (!back && !aligned(p->residual, w->rsz)) || !aligned(p->weight, 4) || !aligned(p->bias, 4))
    return SSCAN_ERR_ALIGN;
  w->x = range_of(p->x, w->empty ? 0 : size_t(e) * xsz);
  w->residual = range_of(back ? nullptr : p->residual, w->res_bytes);
  w->weight = range_of(p->weight, w->vec_bytes);
  w->bias = range_of(p->bias, w->vec_bytes);
  w->a = sscan::LayerNormArgs{};
  w->a.x = p->x;
  w->a.x_stride = p->x_stride;
  w->a.residual = back ? nullptr : p->residual;
  w->a.weight = p->weight;
  w->a.bias = p->bias;
  w->a.rows = p->rows;
  w->a.size = p->size;
  w->a.eps = p->eps;
  w->a.io_bf16 = p->io_dtype == SSCAN_BF16;
  w->a.res_bf16 = p->residual_dtype == SSCAN_BF16;
  return SSCAN_OK;
}

int check_layer(const sscan_layer_norm_params* p, const void* out, const void* total, LayerView* w) {
  const int st = view_layer(p, false, w);
  if (st != SSCAN_OK || w->empty) return st;
  if (!out || (p->residual && !total)) return SSCAN_ERR_NULL;
  if (!aligned(out, w->esz) || !aligned(total, w->rsz)) return SSCAN_ERR_ALIGN;
  const Range o = range_of(out, w->bytes), t = range_of(total, w->res_bytes);
  if (clash(o, {w->x, w->residual, w->weight, w->bias, t}) || clash(t, {w->x, w->weight, w->bias}) ||
      (total != p->residual && overlap(t, w->residual)))
    return SSCAN_ERR_ALIAS;
  return SSCAN_OK;
}

int check_layer_bwd(const sscan_layer_norm_params* p, const void* dout, const void* dtotal, const void* dx,
                    const void* dresidual, const float* dweight, const float* dbias, const void* workspace,
                    size_t workspace_bytes, LayerView* w) {
  int st = view_layer(p, true, w);
  if (st != SSCAN_OK) return st;
  if (!w->empty && (!dout || !dx)) return SSCAN_ERR_NULL;
  if ((dweight && !p->weight) || (dbias && !p->bias)) return SSCAN_ERR_NULL;
  if (!aligned(dout, w->esz) || !aligned(dx, w->esz) || !aligned(dtotal, w->rsz) || !aligned(dresidual, w->rsz) ||
      !aligned(dweight, 4) || !aligned(dbias, 4))
    return SSCAN_ERR_ALIGN;
  const size_t need = w->empty ? 0 : sscan::layer_norm_bwd_workspace(p->rows, p->size);
  st = check_workspace(workspace, workspace_bytes, need, 16);
  if (st != SSCAN_OK) return st;
  const Range d = range_of(dout, w->bytes), dt = range_of(dtotal, w->res_bytes), ws = range_of(workspace, need);
  const Range outs[4] = {range_of(dx, w->bytes), range_of(dresidual, w->res_bytes), range_of(dweight, w->vec_bytes),
                         range_of(dbias, w->vec_bytes)};
  if (clash(ws, {w->x, w->weight, w->bias, d, dt})) return SSCAN_ERR_ALIAS;
  for (int i = 0; i < 4; ++i) {
    if (clash(outs[i], {w->x, w->weight, w->bias, d, ws})) return SSCAN_ERR_ALIAS;
    if (!(i == 1 && dresidual == dtotal) && overlap(outs[i], dt)) return SSCAN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return SSCAN_ERR_ALIAS;
  }
  return SSCAN_OK;
}

}  // namespace

extern "C" {

int sscan_validate_rec_fwd(const sscan_rec_params* p, const void* out, const float* h_last, const sscan_rec_kept* kept,
                           const void* workspace, size_t workspace_bytes) {
  RecView w{};
  return check_rec_fwd(p, out, h_last, kept, workspace, workspace_bytes, &w);
}

int sscan_rec_fwd(const sscan_rec_params* p, void* out, float* h_last, const sscan_rec_kept* kept, void* stream,
                  void* workspace, size_t workspace_bytes) {
  RecView w{};
  const int st = check_rec_fwd(p, out, h_last, kept, workspace, workspace_bytes, &w);
  if (st != SSCAN_OK || w.no_rows) return st;
  w.a.out = out;
  w.a.h_last = h_last;
  return status_of(sscan::launch_rec_fwd(w.a, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

int sscan_validate_rec_step(const sscan_rec_params* p, const float* state, const void* out) {
  RecView w{};
  return check_rec_step(p, state, out, &w);
}

int sscan_rec_step(const sscan_rec_params* p, float* state, void* out, void* stream) {
  RecView w{};
  const int st = check_rec_step(p, state, out, &w);
  if (st != SSCAN_OK || w.no_rows) return st;
  w.a.h0 = state;
  w.a.h_last = state;
  w.a.out = out;
  return status_of(sscan::launch_rec_step(w.a, static_cast<hipStream_t>(stream)));
}

int sscan_validate_rec_bwd(const sscan_rec_params* p, const sscan_rec_kept* kept, const void* dout,
                           const float* dh_last, const sscan_rec_grads* grads, const void* workspace,
                           size_t workspace_bytes) {
  RecView w{};
  return check_rec_bwd(p, kept, dout, dh_last, grads, workspace, workspace_bytes, &w);
}

int sscan_rec_bwd(const sscan_rec_params* p, const sscan_rec_kept* kept, const void* dout, const float* dh_last,
                  const sscan_rec_grads* grads, void* stream, void* workspace, size_t workspace_bytes) {
  RecView w{};
  const int st = check_rec_bwd(p, kept, dout, dh_last, grads, workspace, workspace_bytes, &w);
  // rows of no channels have nothing to differentiate; no rows leave a sum over none
  if (st != SSCAN_OK || p->dim == 0) return st;
  const sscan::RecBwdArgs a{w.a, dout, dh_last, grads->dx, grads->dg, grads->di, grads->dz, grads->dlam, grads->dh0};
  return status_of(sscan::launch_rec_bwd(a, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

size_t sscan_rec_workspace_bytes(int64_t batch, int64_t len, int64_t dim, int io_dtype) {
  return rec_sizes_ok(batch, len, dim, io_dtype) ? sscan::rec_workspace(batch, len, dim, io_dtype == SSCAN_BF16) : 0;
}

size_t sscan_rec_bwd_workspace_bytes(int64_t batch, int64_t len, int64_t dim, int io_dtype) {
  return rec_sizes_ok(batch, len, dim, io_dtype) ? sscan::rec_bwd_workspace(batch, len, dim, io_dtype == SSCAN_BF16) : 0;
}

int sscan_validate_pack8(const void* x, int64_t x_stride, int64_t rows, int64_t size, int io_dtype, const int8_t* q,
                         const float* scale) {
  bool empty = false;
  return check_pack8(x, x_stride, rows, size, io_dtype, q, scale, true, &empty);
}

int sscan_pack8(const void* x, int64_t x_stride, int64_t rows, int64_t size, int io_dtype, int8_t* q, float* scale,
                void* stream) {
  bool empty = false;
  const int st = check_pack8(x, x_stride, rows, size, io_dtype, q, scale, true, &empty);
  if (st != SSCAN_OK || empty) return st;
  const sscan::PackArgs a{x, x_stride, q, scale, nullptr, rows, size, io_dtype == SSCAN_BF16};
  return status_of(sscan::launch_pack8(a, static_cast<hipStream_t>(stream)));
}

int sscan_validate_unpack8(const int8_t* q, const float* scale, int64_t rows, int64_t size, int io_dtype,
                           const void* out) {
  bool empty = false;
  return check_pack8(out, size, rows, size, io_dtype, q, scale, false, &empty);
}

int sscan_unpack8(const int8_t* q, const float* scale, int64_t rows, int64_t size, int io_dtype, void* out,
                  void* stream) {
  bool empty = false;
  const int st = check_pack8(out, size, rows, size, io_dtype, q, scale, false, &empty);
  if (st != SSCAN_OK || empty) return st;
  const sscan::PackArgs a{nullptr, 0, const_cast<int8_t*>(q), const_cast<float*>(scale), out, rows, size,
                          io_dtype == SSCAN_BF16};
  return status_of(sscan::launch_unpack8(a, static_cast<hipStream_t>(stream)));
}

int sscan_validate_layer_norm(const sscan_layer_norm_params* p, const void* out, const void* total) {
  LayerView w{};
  return check_layer(p, out, total, &w);
}

int sscan_layer_norm(const sscan_layer_norm_params* p, void* out, void* total, void* stream) {
  LayerView w{};
  const int st = check_layer(p, out, total, &w);
  if (st != SSCAN_OK || w.empty) return st;
  w.a.out = out;
  w.a.total = total;
  return status_of(sscan::launch_layer_norm(w.a, static_cast<hipStream_t>(stream)));
}

int sscan_validate_layer_norm_bwd(const sscan_layer_norm_params* p, const void* dout, const void* dtotal,
                                  const void* dx, const void* dresidual, const float* dweight, const float* dbias,
                                  const void* workspace, size_t workspace_bytes) {
  LayerView w{};
  return check_layer_bwd(p, dout, dtotal, dx, dresidual, dweight, dbias, workspace, workspace_bytes, &w);
}

int sscan_layer_norm_bwd(const sscan_layer_norm_params* p, const void* dout, const void* dtotal, void* dx,
                         void* dresidual, float* dweight, float* dbias, void* stream, void* workspace,
                         size_t workspace_bytes) {
  LayerView w{};
  const int st = check_layer_bwd(p, dout, dtotal, dx, dresidual, dweight, dbias, workspace, workspace_bytes, &w);
  if (st != SSCAN_OK) return st;
  w.a.dout = dout;
  w.a.dtotal = dtotal;
  w.a.dx = dx;
  w.a.dresidual = dresidual;
  w.a.dweight = dweight;
  w.a.dbias = dbias;
  return status_of(
      sscan::launch_layer_norm_bwd(w.a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

size_t sscan_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t size) {
  if (rows <= 0 || size < 1 || size > sscan::kNormMaxSize || product({rows, size}) < 0) return 0;
  return sscan::layer_norm_bwd_workspace(rows, size);
}

}  // extern "C"
