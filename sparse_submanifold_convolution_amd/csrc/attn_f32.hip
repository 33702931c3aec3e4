// Cross attention kernels for float elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_fwd<float>(const Params& p, const FwdPlan& f, hipStream_t s) {
  return launch_fwd_impl<float>(p, f, s);
}
template <>
int launch_bwd<float>(Params p, const BwdPlan& b, float* part_q, float* part_k, float* part_v, uint32_t* bound,
                    hipStream_t s) {
  return launch_bwd_impl<float>(p, b, part_q, part_k, part_v, bound, s);
}

}  // namespace attn
}  // namespace ssc
