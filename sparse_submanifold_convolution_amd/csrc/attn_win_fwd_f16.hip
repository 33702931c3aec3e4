// Windowed attention, forward kernels for _Float16 elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_win_fwd<_Float16>(const Params& p, const FwdPlan& f, hipStream_t s) {
  return launch_fwd_impl<_Float16, true>(p, f, s);
}

}  // namespace attn
}  // namespace ssc
