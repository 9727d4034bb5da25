// gn_join_bwd_mixed.hip -- gn_join_bwd.hpp of a 16-bit type with the stream in fp32.
#include "gn_join_bwd.hpp"

namespace gn {

hipError_t launch_join_bwd_mixed(const JoinBwdArgs& a, int x_dtype, const JoinPlan& p, hipStream_t st)
{
    return x_dtype == GN_BF16 ? one<uint16_t, float, 4>(a, p, st) : one<_Float16, float, 4>(a, p, st);
}

}  // namespace gn
