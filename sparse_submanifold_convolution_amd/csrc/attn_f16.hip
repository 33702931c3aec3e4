// Cross attention kernels for _Float16 elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_fwd<_Float16>(const Params& p, const FwdPlan& f, hipStream_t s) {
  return launch_fwd_impl<_Float16>(p, f, s);
}
template <>
int launch_bwd<_Float16>(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s) {
  return launch_bwd_impl<_Float16>(p, b, w, s);
}

}  // namespace attn
}  // namespace ssc
