// Cross attention kernels for __bf16 elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_fwd<__bf16>(const Params& p, const FwdPlan& f, hipStream_t s) {
  return launch_fwd_impl<__bf16>(p, f, s);
}
template <>
int launch_bwd<__bf16>(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s) {
  return launch_bwd_impl<__bf16>(p, b, w, s);
}

}  // namespace attn
}  // namespace ssc
