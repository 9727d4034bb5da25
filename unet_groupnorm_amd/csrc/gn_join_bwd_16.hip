// gn_join_bwd_16.hip -- gn_join_bwd.hpp where every tensor is of one 16-bit type.
#include "gn_join_bwd.hpp"

namespace gn {

hipError_t launch_join_bwd_16(const JoinBwdArgs& a, int x_dtype, const JoinPlan& p, hipStream_t st)
{
    return x_dtype == GN_BF16 ? one<uint16_t, uint16_t, 8>(a, p, st) : one<_Float16, _Float16, 8>(a, p, st);
}

}  // namespace gn
