// sscan_rec_bwd.hip -- gradients of the gated recurrence (sscan_rec_bwd.h).
#include "sscan_rec_bwd.h"

namespace sscan {
namespace rec {

// Without tokens the adjoint of the last state is that of the entry state.
__global__ __launch_bounds__(256) void through_kernel(const float* from, float* to, int64_t n, float* zeros, int64_t m) {
  const int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (to && k < n) to[k] = from ? from[k] : 0.0f;
  if (zeros && k < m) zeros[k] = 0.0f;
}

}  // namespace rec

size_t rec_bwd_workspace(int64_t batch, int64_t len, int64_t dim, bool io_bf16) {
  if (len == 0) return 0;
  // whichever of the inputs themselves and what was kept of them needs more
  const size_t x = rec::back_plan(batch, len, dim, false, io_bf16).bytes, k = rec::back_plan(batch, len, dim, true, io_bf16).bytes;
  return x > k ? x : k;
}

hipError_t launch_rec_bwd(const RecBwdArgs& w, char* workspace, hipStream_t stream) {
  const RecArgs& a = w.f;
  if (a.len == 0 || a.batch == 0) {
    const int64_t n = a.batch * a.dim, m = n > a.dim ? n : a.dim;
    rec::through_kernel<<<dim3(unsigned(rec::up(m, 256))), 256, 0, stream>>>(w.dh_last, w.dh0, n, w.dlam, a.dim);
    return hipGetLastError();
  }
  const bool kept = a.kept.x != nullptr;
  const rec::BackPlan p = rec::back_plan(a.batch, a.len, a.dim, kept, a.io_bf16);
  if (kept) return rec::launch_bwd_kept(w, p, workspace, stream);
  return rec::by_lane(p.c, a.io_bf16, [&](auto io, auto c) {
    return rec::bwd<decltype(io), decltype(c)::value, false>(w, p, workspace, stream);
  });
}

}  // namespace sscan
