// sscan_rec_keep.hip -- the recurrence's forward pass that leaves its inputs in 8 bits for the
// backward pass, in the same pass over them.
#include "sscan_rec_fwd.h"

namespace sscan {
namespace rec {

hipError_t launch_keep(const RecArgs& a, const Plan& plan, char* workspace, hipStream_t stream) {
  return by_lane(plan.c, a.io_bf16, [&](auto io, auto c) {
    return fwd<decltype(io), decltype(c)::value, true>(a, plan, workspace, stream);
  });
}

}  // namespace rec
}  // namespace sscan
