// sscan_rec_bwd_kept.hip -- gradients of the gated recurrence from inputs that were kept in 8 bits.
#include "sscan_rec_bwd.h"

namespace sscan {
namespace rec {

hipError_t launch_bwd_kept(const RecBwdArgs& w, const BackPlan& plan, char* workspace, hipStream_t stream) {
  if (plan.c == 4) return bwd<bf16, 4, true>(w, plan, workspace, stream);
  return by_lane(plan.c, w.f.io_bf16, [&](auto io, auto c) {
    return bwd<decltype(io), decltype(c)::value, true>(w, plan, workspace, stream);
  });
}

}  // namespace rec
}  // namespace sscan
