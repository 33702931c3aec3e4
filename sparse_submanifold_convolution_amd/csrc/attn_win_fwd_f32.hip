// Windowed attention, forward kernels for float elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_win_fwd<float>(const Params& p, const FwdPlan& f, hipStream_t s) {
  return launch_fwd_impl<float, true>(p, f, s);
}

}  // namespace attn
}  // namespace ssc
