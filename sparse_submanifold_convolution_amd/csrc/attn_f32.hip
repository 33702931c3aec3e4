// Cross attention kernels for float elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_fwd<float>(const Params& p, const FwdPlan& f, hipStream_t s) {
  return launch_fwd_impl<float>(p, f, s);
}
template <>
int launch_bwd<float>(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s) {
  return launch_bwd_impl<float>(p, b, w, s);
}

}  // namespace attn
}  // namespace ssc
