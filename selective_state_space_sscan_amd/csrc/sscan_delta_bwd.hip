#include "sscan_delta.h"
namespace sscan {
DeltaBwdPlan make_delta_bwd_plan(int64_t, int64_t, int, int, int, int, bool) { return DeltaBwdPlan{}; }
hipError_t launch_delta_bwd(const DeltaBwdArgs&, const DeltaBwdPlan&, char*, hipStream_t) { return hipErrorNotSupported; }
}
