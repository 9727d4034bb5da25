// gn_join_bwd_f32.hip -- gn_join_bwd.hpp in fp32.
#include "gn_join_bwd.hpp"

namespace gn {

hipError_t launch_join_bwd_f32(const JoinBwdArgs& a, const JoinPlan& p, hipStream_t st) { return one<float, float, 4>(a, p, st); }

}  // namespace gn
