// sscan_delta_capi.cpp -- C ABI of the gated delta rule and of the norms around a
// mixer: argument checks, then one call into the kernel launchers.  Every check comes
// before any HIP call, so the validate entry points work without a GPU.
#include "sscan.h"

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "sscan_delta.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

Range range_of(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return p ? Range{lo, lo + bytes} : Range{0, 0};
}

bool overlap(const Range& a, const Range& b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

bool clash(const Range& out, std::initializer_list<Range> others) {
  for (const Range& r : others)
    if (overlap(out, r)) return true;
  return false;
}

constexpr int64_t kMaxElems = int64_t(1) << 50;

// a * b * ..., or -1 beyond 2^50.
int64_t product(std::initializer_list<int64_t> f) {
  int64_t n = 1;
  for (int64_t x : f)
    if (__builtin_mul_overflow(n, x, &n) || n > kMaxElems) return -1;
  return n;
}

// Elements from the first to one past the last of a strided view whose last `size`
// elements are contiguous, or -1 (a negative stride, or beyond 2^50).
int64_t extent(const int64_t* dims, const int64_t* strides, int n, int64_t size) {
  int64_t last = size;
  for (int i = 0; i < n; ++i) {
    if (strides[i] < 0) return -1;
    if (dims[i] <= 1) continue;
    int64_t step = 0;
    if (__builtin_mul_overflow(dims[i] - 1, strides[i], &step) || __builtin_add_overflow(last, step, &last) ||
        last > kMaxElems)
      return -1;
  }
  return last;
}

bool dtype_ok(int d) { return d == SSCAN_F32 || d == SSCAN_BF16; }
size_t dtype_size(int d) { return d == SSCAN_BF16 ? 2 : 4; }

sscan::DeltaStride stride_of(const int64_t* s) { return sscan::DeltaStride{s[0], s[1], s[2]}; }

struct DeltaView {
  sscan::DeltaArgs a;
  size_t esz;
  size_t state_bytes, qk_bytes, v_bytes, gate_bytes;  // contiguous tensors of these shapes
  Range q, k, v, g, beta, lengths, h0;
  bool no_rows, no_tokens;
};

// Sizes, codes, pointers and strides of the inputs, and the ranges they cover.
int view_delta(const sscan_delta_params* p, DeltaView* w) {
  if (!p) return SSCAN_ERR_NULL;
  if (p->batch < 0 || p->len < 0 || p->qk_heads < 0 || p->v_heads < 0) return SSCAN_ERR_SHAPE;
  if (!dtype_ok(p->io_dtype) || (p->qk_norm != 0 && p->qk_norm != 1) || !std::isfinite(p->scale))
    return SSCAN_ERR_UNSUPPORTED;
  if (p->dk < 1 || p->dk > sscan::kDeltaMaxK || p->dv < 1 || p->dv > sscan::kDeltaMaxV) return SSCAN_ERR_UNSUPPORTED;
  w->no_rows = p->batch == 0 || p->v_heads == 0;
  w->no_tokens = p->len == 0;
  if (p->v_heads > 0 && (p->qk_heads < 1 || p->v_heads % p->qk_heads != 0)) return SSCAN_ERR_SHAPE;
  if (w->no_rows) return SSCAN_OK;
  // tokens are counted in 32 bits; the grids (a block per chunk and head, at most four
  // per head's columns) stay below 2^24 blocks of 256 threads
  const int64_t chunks = (p->len + sscan::kDeltaChunk - 1) / sscan::kDeltaChunk;
  if (p->len > (int64_t(1) << 30) || p->v_heads > (1 << 20)) return SSCAN_ERR_SHAPE;
  const int64_t blocks = product({p->batch, p->v_heads, chunks > 4 ? chunks : 4});
  if (blocks < 0 || blocks >= (int64_t(1) << 24)) return SSCAN_ERR_SHAPE;
  const int64_t n_state = product({p->batch, p->v_heads, p->dk, p->dv}),
                n_qk = product({p->batch, p->len, p->qk_heads, p->dk}),
                n_v = product({p->batch, p->len, p->v_heads, p->dv}), n_g = product({p->batch, p->len, p->v_heads});
  if (n_state < 0 || n_qk < 0 || n_v < 0 || n_g < 0) return SSCAN_ERR_SHAPE;
  w->esz = dtype_size(p->io_dtype);
  w->state_bytes = size_t(n_state) * 4;
  w->qk_bytes = size_t(n_qk) * w->esz;
  w->v_bytes = size_t(n_v) * w->esz;
  w->gate_bytes = size_t(n_g) * 4;
  if (!w->no_tokens && (!p->q || !p->k || !p->v || !p->g || !p->beta)) return SSCAN_ERR_NULL;
  if (!aligned(p->q, w->esz) || !aligned(p->k, w->esz) || !aligned(p->v, w->esz) || !aligned(p->g, 4) ||
      !aligned(p->beta, 4) || !aligned(p->lengths, 4) || !aligned(p->h0, 16))
    return SSCAN_ERR_ALIGN;
  // a chunk's rows are addressed by 32-bit byte offsets; a single token's stride is never
  // used
  if (p->v_heads * p->dv >= sscan::kDeltaMaxStride || p->qk_heads * p->dk >= sscan::kDeltaMaxStride)
    return SSCAN_ERR_UNSUPPORTED;
  if (p->len > 1 && (p->q_stride[1] >= sscan::kDeltaMaxStride || p->k_stride[1] >= sscan::kDeltaMaxStride ||
                     p->v_stride[1] >= sscan::kDeltaMaxStride))
    return SSCAN_ERR_UNSUPPORTED;
  const int64_t qd[3] = {p->batch, p->len, p->qk_heads}, vd[3] = {p->batch, p->len, p->v_heads};
  const int64_t eq = extent(qd, p->q_stride, 3, p->dk), ek = extent(qd, p->k_stride, 3, p->dk),
                ev = extent(vd, p->v_stride, 3, p->dv), eg = extent(vd, p->g_stride, 3, 1),
                eb = extent(vd, p->beta_stride, 3, 1);
  if (eq < 0 || ek < 0 || ev < 0 || eg < 0 || eb < 0) return SSCAN_ERR_SHAPE;
  const size_t live = w->no_tokens ? 0 : 1;
  w->q = range_of(p->q, live * size_t(eq) * w->esz);
  w->k = range_of(p->k, live * size_t(ek) * w->esz);
  w->v = range_of(p->v, live * size_t(ev) * w->esz);
  w->g = range_of(p->g, live * size_t(eg) * 4);
  w->beta = range_of(p->beta, live * size_t(eb) * 4);
  w->lengths = range_of(p->lengths, size_t(p->batch) * 4);
  w->h0 = range_of(p->h0, w->state_bytes);
  w->a = sscan::DeltaArgs{p->q, p->k, p->v, p->g, p->beta, stride_of(p->q_stride), stride_of(p->k_stride),
                          stride_of(p->v_stride), stride_of(p->g_stride), stride_of(p->beta_stride), p->lengths,
                          p->h0, nullptr, nullptr, p->batch, p->len, int(p->qk_heads), int(p->v_heads), int(p->dk),
                          int(p->dv), p->scale, p->qk_norm, p->io_dtype == SSCAN_BF16};
  if (p->len <= 1) {
    w->a.sq.t = w->a.sk.t = p->dk;
    w->a.sv.t = p->dv;
  }
  return SSCAN_OK;
}

int check_workspace(const void* workspace, size_t have, size_t need, size_t align) {
  if (need == 0) return SSCAN_OK;
  if (!workspace || have < need) return SSCAN_ERR_WORKSPACE;
  return aligned(workspace, align) ? SSCAN_OK : SSCAN_ERR_ALIGN;
}

sscan::DeltaPlan plan_of(const sscan_delta_params* p) {
  return sscan::make_delta_plan(p->batch, p->len, int(p->qk_heads), int(p->v_heads), int(p->dk), int(p->dv),
                                p->io_dtype == SSCAN_BF16);
}

sscan::DeltaBwdPlan bwd_plan_of(const sscan_delta_params* p) {
  return sscan::make_delta_bwd_plan(p->batch, p->len, int(p->qk_heads), int(p->v_heads), int(p->dk), int(p->dv),
                                    p->io_dtype == SSCAN_BF16);
}

int check_delta_fwd(const sscan_delta_params* p, const void* out, const float* h_last, const void* workspace,
                    size_t workspace_bytes, DeltaView* w, sscan::DeltaPlan* plan) {
  int st = view_delta(p, w);
  if (st != SSCAN_OK || w->no_rows) return st;
  if (!h_last || (!w->no_tokens && !out)) return SSCAN_ERR_NULL;
  if (!aligned(h_last, 16) || !aligned(out, w->esz)) return SSCAN_ERR_ALIGN;
  *plan = plan_of(p);
  st = check_workspace(workspace, workspace_bytes, plan->workspace_bytes, 256);
  if (st != SSCAN_OK) return st;
  const Range o = range_of(out, w->v_bytes), s = range_of(h_last, w->state_bytes);
  const Range ws = range_of(workspace, plan->workspace_bytes);
  if (clash(o, {w->q, w->k, w->v, w->g, w->beta, w->lengths, w->h0, s, ws}) ||
      clash(s, {w->q, w->k, w->v, w->g, w->beta, w->lengths, ws}) || (h_last != p->h0 && overlap(s, w->h0)))
    return SSCAN_ERR_ALIAS;
  return SSCAN_OK;
}

int check_delta_step(const sscan_delta_params* p, const float* state, const void* out, DeltaView* w) {
  if (!p) return SSCAN_ERR_NULL;
  if (p->len != 1) return SSCAN_ERR_SHAPE;
  if (p->h0) return SSCAN_ERR_UNSUPPORTED;
  sscan::DeltaPlan plan{};
  return check_delta_fwd(p, out, state, nullptr, 0, w, &plan);
}

int check_delta_bwd(const sscan_delta_params* p, const void* dout, const float* dh_last,
                    const sscan_delta_grads* grads, const void* workspace, size_t workspace_bytes, DeltaView* w,
                    sscan::DeltaBwdPlan* plan) {
  if (!grads) return SSCAN_ERR_NULL;
  int st = view_delta(p, w);
  if (st != SSCAN_OK || w->no_rows) return st;
  const sscan_delta_grads& g = *grads;
  if (!w->no_tokens && (!dout || !g.dq || !g.dk || !g.dv || !g.dg || !g.dbeta)) return SSCAN_ERR_NULL;
  if (!aligned(dout, w->esz) || !aligned(g.dq, w->esz) || !aligned(g.dk, w->esz) || !aligned(g.dv, w->esz) ||
      !aligned(g.dg, 4) || !aligned(g.dbeta, 4) || !aligned(g.dh0, 4) || !aligned(dh_last, 4))
    return SSCAN_ERR_ALIGN;
  *plan = bwd_plan_of(p);
  st = check_workspace(workspace, workspace_bytes, plan->workspace_bytes, 256);
  if (st != SSCAN_OK) return st;
  const Range outs[6] = {range_of(g.dq, w->qk_bytes), range_of(g.dk, w->qk_bytes),  range_of(g.dv, w->v_bytes),
                         range_of(g.dg, w->gate_bytes), range_of(g.dbeta, w->gate_bytes),
                         range_of(g.dh0, w->state_bytes)};
  const Range ws = range_of(workspace, plan->workspace_bytes), d = range_of(dout, w->v_bytes),
              dh = range_of(dh_last, w->state_bytes);
  for (int i = 0; i < 6; ++i) {
    if (clash(outs[i], {w->q, w->k, w->v, w->g, w->beta, w->lengths, w->h0, d, dh, ws})) return SSCAN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return SSCAN_ERR_ALIAS;
  }
  return SSCAN_OK;
}

// The sizes a workspace or plan query is asked for, as the call itself checks them.
int check_delta_sizes(int64_t batch, int64_t len, int64_t hk, int64_t hv, int64_t dk, int64_t dv, int io_dtype,
                      sscan_delta_params* p, bool* no_rows) {
  *p = sscan_delta_params{};
  p->batch = batch;
  p->len = len;
  p->qk_heads = hk;
  p->v_heads = hv;
  p->dk = dk;
  p->dv = dv;
  p->io_dtype = io_dtype;
  DeltaView w{};
  const int st = view_delta(p, &w);
  *no_rows = w.no_rows;
  return st == SSCAN_ERR_NULL ? SSCAN_OK : st;  // there are no pointers to check
}

bool delta_sizes_ok(int64_t batch, int64_t len, int64_t hk, int64_t hv, int64_t dk, int64_t dv, int io_dtype,
                    sscan_delta_params* p) {
  bool no_rows = false;
  return check_delta_sizes(batch, len, hk, hv, dk, dv, io_dtype, p, &no_rows) == SSCAN_OK && !no_rows;
}

struct GatedView {
  sscan::GatedNormArgs a;
  size_t esz, bytes, weight_bytes;
  Range x, z, weight;
  bool empty;
};

int view_gated(const sscan_gated_norm_params* p, GatedView* w) {
  if (!p) return SSCAN_ERR_NULL;
  if (p->rows < 0 || p->heads < 0) return SSCAN_ERR_SHAPE;
  if (p->size < 1 || p->size > sscan::kNormMaxSize || !dtype_ok(p->io_dtype) ||
      (p->gate_first != 0 && p->gate_first != 1) || (p->per_head != 0 && p->per_head != 1) ||
      !std::isfinite(p->eps) || p->eps < 0)
    return SSCAN_ERR_UNSUPPORTED;
  // a block or more for each head whose weight's gradient is summed
  if (p->per_head && p->heads > sscan::kNormMaxHeads) return SSCAN_ERR_SHAPE;
  w->empty = p->rows == 0 || p->heads == 0;
  const int64_t n = product({p->rows, p->heads, p->size}), nw = p->size * (p->per_head ? p->heads : 1);
  if (n < 0) return SSCAN_ERR_SHAPE;
  w->esz = dtype_size(p->io_dtype);
  w->bytes = size_t(n) * w->esz;
  w->weight_bytes = size_t(nw) * 4;
  if (!w->empty && (!p->x || !p->z)) return SSCAN_ERR_NULL;
  if (p->per_head && nw > 0 && !p->weight) return SSCAN_ERR_NULL;
  if (!aligned(p->x, w->esz) || !aligned(p->z, w->esz) || !aligned(p->weight, 4)) return SSCAN_ERR_ALIGN;
  const int64_t dims[2] = {p->rows, p->heads};
  const int64_t ex = extent(dims, p->x_stride, 2, p->size), ez = extent(dims, p->z_stride, 2, p->size);
  if (ex < 0 || ez < 0) return SSCAN_ERR_SHAPE;
  w->x = range_of(p->x, w->empty ? 0 : size_t(ex) * w->esz);
  w->z = range_of(p->z, w->empty ? 0 : size_t(ez) * w->esz);
  w->weight = range_of(p->weight, w->weight_bytes);
  w->a = sscan::GatedNormArgs{p->x, p->z, p->x_stride[0], p->x_stride[1], p->z_stride[0], p->z_stride[1], p->weight,
                              p->per_head, nullptr, nullptr, nullptr, nullptr, nullptr, p->rows, p->heads, p->size,
                              p->eps, p->gate_first, p->io_dtype == SSCAN_BF16};
  return SSCAN_OK;
}

int check_gated(const sscan_gated_norm_params* p, const void* out, GatedView* w) {
  const int st = view_gated(p, w);
  if (st != SSCAN_OK || w->empty) return st;
  if (!out) return SSCAN_ERR_NULL;
  if (!aligned(out, w->esz)) return SSCAN_ERR_ALIGN;
  return clash(range_of(out, w->bytes), {w->x, w->z, w->weight}) ? SSCAN_ERR_ALIAS : SSCAN_OK;
}

int check_gated_bwd(const sscan_gated_norm_params* p, const void* dout, const void* dx, const void* dz,
                    const float* dweight, const void* workspace, size_t workspace_bytes, GatedView* w) {
  int st = view_gated(p, w);
  if (st != SSCAN_OK) return st;
  if (dweight && !p->weight) return SSCAN_ERR_NULL;
  if (!w->empty && (!dout || !dx || !dz)) return SSCAN_ERR_NULL;
  if (!aligned(dout, w->esz) || !aligned(dx, w->esz) || !aligned(dz, w->esz) || !aligned(dweight, 4))
    return SSCAN_ERR_ALIGN;
  const size_t need = w->empty ? 0 : sscan::gated_norm_bwd_workspace(p->rows, p->heads, p->size);
  st = check_workspace(workspace, workspace_bytes, need, 16);
  if (st != SSCAN_OK) return st;
  const Range d = range_of(dout, w->bytes), ws = range_of(workspace, need);
  const Range outs[3] = {range_of(dx, w->bytes), range_of(dz, w->bytes), range_of(dweight, w->weight_bytes)};
  for (int i = 0; i < 3; ++i) {
    if (clash(outs[i], {w->x, w->z, w->weight, d, ws})) return SSCAN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return SSCAN_ERR_ALIAS;
  }
  return SSCAN_OK;
}

struct AddView {
  sscan::AddNormArgs a;
  size_t esz, rsz, bytes, res_bytes, vec_bytes;
  Range x, residual, weight, scale, post;
  bool empty;
};

int view_add(const sscan_add_norm_params* p, AddView* w) {
  if (!p) return SSCAN_ERR_NULL;
  if (p->rows < 0) return SSCAN_ERR_SHAPE;
  if (p->size < 1 || p->size > sscan::kNormMaxSize || !dtype_ok(p->io_dtype) || !dtype_ok(p->residual_dtype) ||
      !std::isfinite(p->eps) || p->eps < 0)
    return SSCAN_ERR_UNSUPPORTED;
  w->empty = p->rows == 0;
  const int64_t n = product({p->rows, p->size});
  if (n < 0) return SSCAN_ERR_SHAPE;
  w->esz = dtype_size(p->io_dtype);
  w->rsz = dtype_size(p->residual_dtype);
  w->bytes = size_t(n) * w->esz;
  w->res_bytes = size_t(n) * w->rsz;
  w->vec_bytes = size_t(p->size) * 4;
  if (!w->empty && !p->x) return SSCAN_ERR_NULL;
  if (!aligned(p->x, w->esz) || !aligned(p->residual, w->rsz) || !aligned(p->weight, 4) || !aligned(p->scale, 4) ||
      !aligned(p->post_weight, 4))
    return SSCAN_ERR_ALIGN;
  w->x = range_of(p->x, w->bytes);
  w->residual = range_of(p->residual, w->res_bytes);
  w->weight = range_of(p->weight, w->vec_bytes);
  w->scale = range_of(p->scale, w->vec_bytes);
  w->post = range_of(p->post_weight, w->vec_bytes);
  w->a = sscan::AddNormArgs{p->x, p->residual, p->weight, p->scale, p->post_weight, nullptr, nullptr, nullptr,
                            nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, p->rows, p->size, p->eps,
                            p->io_dtype == SSCAN_BF16, p->residual_dtype == SSCAN_BF16};
  return SSCAN_OK;
}

int check_add(const sscan_add_norm_params* p, const void* out, const void* residual_out, AddView* w) {
  const int st = view_add(p, w);
  if (st != SSCAN_OK || w->empty) return st;
  if (!out || !residual_out) return SSCAN_ERR_NULL;
  if (!aligned(out, w->esz) || !aligned(residual_out, w->rsz)) return SSCAN_ERR_ALIGN;
  const Range o = range_of(out, w->bytes), r = range_of(residual_out, w->res_bytes);
  if (clash(o, {w->x, w->residual, w->weight, w->scale, w->post, r}) || clash(r, {w->x, w->weight, w->scale, w->post}) ||
      (residual_out != p->residual && overlap(r, w->residual)))
    return SSCAN_ERR_ALIAS;
  return SSCAN_OK;
}

int check_add_bwd(const sscan_add_norm_params* p, const void* dout, const void* dresidual_out, const void* dx,
                  const void* dresidual, const float* dweight, const float* dscale, const float* dpost_weight,
                  const void* workspace, size_t workspace_bytes, AddView* w) {
  int st = view_add(p, w);
  if (st != SSCAN_OK) return st;
  if (!w->empty && (!p->residual || !dout || !dx || !dresidual)) return SSCAN_ERR_NULL;
  if ((dweight && !p->weight) || (dscale && !p->scale) || (dpost_weight && !p->post_weight)) return SSCAN_ERR_NULL;
  if (!aligned(dout, w->esz) || !aligned(dx, w->esz) || !aligned(dresidual_out, w->rsz) ||
      !aligned(dresidual, w->rsz) || !aligned(dweight, 4) || !aligned(dscale, 4) || !aligned(dpost_weight, 4))
    return SSCAN_ERR_ALIGN;
  const size_t need = w->empty ? 0 : sscan::add_norm_bwd_workspace(p->rows, p->size);
  st = check_workspace(workspace, workspace_bytes, need, 16);
  if (st != SSCAN_OK) return st;
  const Range d = range_of(dout, w->bytes), dr = range_of(dresidual_out, w->res_bytes), ws = range_of(workspace, need);
  const Range outs[5] = {range_of(dx, w->bytes), range_of(dresidual, w->res_bytes), range_of(dweight, w->vec_bytes),
                         range_of(dscale, w->vec_bytes), range_of(dpost_weight, w->vec_bytes)};
  for (int i = 0; i < 5; ++i) {
    if (clash(outs[i], {w->x, w->residual, w->weight, w->scale, w->post, d, ws})) return SSCAN_ERR_ALIAS;
    if (!(i == 1 && dresidual == dresidual_out) && overlap(outs[i], dr)) return SSCAN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return SSCAN_ERR_ALIAS;
  }
  return SSCAN_OK;
}

int status_of(hipError_t e) { return e == hipSuccess ? SSCAN_OK : SSCAN_ERR_HIP; }

}  // namespace

extern "C" {

int sscan_validate_delta_fwd(const sscan_delta_params* p, const void* out, const float* h_last, const void* workspace,
                             size_t workspace_bytes) {
  DeltaView w{};
  sscan::DeltaPlan plan{};
  return check_delta_fwd(p, out, h_last, workspace, workspace_bytes, &w, &plan);
}

int sscan_delta_fwd(const sscan_delta_params* p, void* out, float* h_last, void* stream, void* workspace,
                    size_t workspace_bytes) {
  DeltaView w{};
  sscan::DeltaPlan plan{};
  const int st = check_delta_fwd(p, out, h_last, workspace, workspace_bytes, &w, &plan);
  if (st != SSCAN_OK || w.no_rows) return st;
  w.a.out = out;
  w.a.h_last = h_last;
  return status_of(
      sscan::launch_delta_fwd(w.a, plan, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

int sscan_validate_delta_step(const sscan_delta_params* p, const float* state, const void* out) {
  DeltaView w{};
  return check_delta_step(p, state, out, &w);
}

int sscan_delta_step(const sscan_delta_params* p, float* state, void* out, void* stream) {
  DeltaView w{};
  const int st = check_delta_step(p, state, out, &w);
  if (st != SSCAN_OK || w.no_rows) return st;
  w.a.h0 = state;
  w.a.h_last = state;
  w.a.out = out;
  return status_of(sscan::launch_delta_fwd(w.a, plan_of(p), nullptr, static_cast<hipStream_t>(stream)));
}

int sscan_validate_delta_bwd(const sscan_delta_params* p, const void* dout, const float* dh_last,
                             const sscan_delta_grads* grads, const void* workspace, size_t workspace_bytes) {
  DeltaView w{};
  sscan::DeltaBwdPlan plan{};
  return check_delta_bwd(p, dout, dh_last, grads, workspace, workspace_bytes, &w, &plan);
}

int sscan_delta_bwd(const sscan_delta_params* p, const void* dout, const float* dh_last,
                    const sscan_delta_grads* grads, void* stream, void* workspace, size_t workspace_bytes) {
  DeltaView w{};
  sscan::DeltaBwdPlan plan{};
  const int st = check_delta_bwd(p, dout, dh_last, grads, workspace, workspace_bytes, &w, &plan);
  if (st != SSCAN_OK || w.no_rows) return st;
  const sscan::DeltaBwdArgs a{w.a, dout, dh_last, grads->dq, grads->dk, grads->dv, grads->dg, grads->dbeta, grads->dh0};
  return status_of(sscan::launch_delta_bwd(a, plan, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
}

size_t sscan_delta_workspace_bytes(int64_t batch, int64_t len, int64_t qk_heads, int64_t v_heads, int64_t dk,
                                   int64_t dv, int io_dtype) {
  sscan_delta_params p;
  return delta_sizes_ok(batch, len, qk_heads, v_heads, dk, dv, io_dtype, &p) ? plan_of(&p).workspace_bytes : 0;
}

size_t sscan_delta_bwd_workspace_bytes(int64_t batch, int64_t len, int64_t qk_heads, int64_t v_heads, int64_t dk,
                                       int64_t dv, int io_dtype) {
  sscan_delta_params p;
  return delta_sizes_ok(batch, len, qk_heads, v_heads, dk, dv, io_dtype, &p) ? bwd_plan_of(&p).workspace_bytes : 0;
}

int sscan_delta_plan(int64_t batch, int64_t len, int64_t qk_heads, int64_t v_heads, int64_t dk, int64_t dv,
                     int io_dtype, int64_t* out) {
  if (!out) return SSCAN_ERR_NULL;
  sscan_delta_params p;
  bool no_rows = false;
  const int st = check_delta_sizes(batch, len, qk_heads, v_heads, dk, dv, io_dtype, &p, &no_rows);
  if (st != SSCAN_OK) return st;
  const sscan::DeltaPlan plan = no_rows ? sscan::DeltaPlan{} : plan_of(&p);
  out[0] = plan.recurrent ? 0 : plan.nchunk;
  out[1] = plan.nseg;
  out[2] = plan.seg_chunks;
  out[3] = plan.waves;
  return SSCAN_OK;
}

int sscan_validate_gated_norm(const sscan_gated_norm_params* p, const void* out) {
  GatedView w{};
  return check_gated(p, out, &w);
}

int sscan_gated_norm(const sscan_gated_norm_params* p, void* out, void* stream) {
  GatedView w{};
  const int st = check_gated(p, out, &w);
  if (st != SSCAN_OK || w.empty) return st;
  w.a.out = out;
  return status_of(sscan::launch_gated_norm(w.a, static_cast<hipStream_t>(stream)));
}

int sscan_validate_gated_norm_bwd(const sscan_gated_norm_params* p, const void* dout, const void* dx, const void* dz,
                                  const float* dweight, const void* workspace, size_t workspace_bytes) {
  GatedView w{};
  return check_gated_bwd(p, dout, dx, dz, dweight, workspace, workspace_bytes, &w);
}

int sscan_gated_norm_bwd(const sscan_gated_norm_params* p, const void* dout, void* dx, void* dz, float* dweight,
                         void* stream, void* workspace, size_t workspace_bytes) {
  GatedView w{};
  const int st = check_gated_bwd(p, dout, dx, dz, dweight, workspace, workspace_bytes, &w);
  if (st != SSCAN_OK) return st;
  w.a.dout = dout;
  w.a.dx = dx;
  w.a.dz = dz;
  w.a.dweight = dweight;
  return status_of(
      sscan::launch_gated_norm_bwd(w.a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

size_t sscan_gated_norm_bwd_workspace_bytes(int64_t rows, int64_t heads, int64_t size) {
  if (rows <= 0 || heads <= 0 || size < 1 || size > sscan::kNormMaxSize || product({rows, heads, size}) < 0) return 0;
  return sscan::gated_norm_bwd_workspace(rows, heads, size);
}

int sscan_validate_add_norm(const sscan_add_norm_params* p, const void* out, const void* residual_out) {
  AddView w{};
  return check_add(p, out, residual_out, &w);
}

int sscan_add_norm(const sscan_add_norm_params* p, void* out, void* residual_out, void* stream) {
  AddView w{};
  const int st = check_add(p, out, residual_out, &w);
  if (st != SSCAN_OK || w.empty) return st;
  w.a.out = out;
  w.a.residual_out = residual_out;
  return status_of(sscan::launch_add_norm(w.a, static_cast<hipStream_t>(stream)));
}

int sscan_validate_add_norm_bwd(const sscan_add_norm_params* p, const void* dout, const void* dresidual_out,
                                const void* dx, const void* dresidual, const float* dweight, const float* dscale,
                                const float* dpost_weight, const void* workspace, size_t workspace_bytes) {
  AddView w{};
  return check_add_bwd(p, dout, dresidual_out, dx, dresidual, dweight, dscale, dpost_weight, workspace,
                       workspace_bytes, &w);
}

int sscan_add_norm_bwd(const sscan_add_norm_params* p, const void* dout, const void* dresidual_out, void* dx,
                       void* dresidual, float* dweight, float* dscale, float* dpost_weight, void* stream,
                       void* workspace, size_t workspace_bytes) {
  AddView w{};
  const int st = check_add_bwd(p, dout, dresidual_out, dx, dresidual, dweight, dscale, dpost_weight, workspace,
                               workspace_bytes, &w);
  if (st != SSCAN_OK) return st;
  w.a.dout = dout;
  w.a.dresidual_out = dresidual_out;
  w.a.dx = dx;
  w.a.dresidual = dresidual;
  w.a.dweight = dweight;
  w.a.dscale = dscale;
  w.a.dpost_weight = dpost_weight;
  return status_of(sscan::launch_add_norm_bwd(w.a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

size_t sscan_add_norm_bwd_workspace_bytes(int64_t rows, int64_t size) {
  if (rows <= 0 || size < 1 || size > sscan::kNormMaxSize || product({rows, size}) < 0) return 0;
  return sscan::add_norm_bwd_workspace(rows, size);
}

}  // extern "C"
