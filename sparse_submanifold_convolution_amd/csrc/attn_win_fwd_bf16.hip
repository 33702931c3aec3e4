// Windowed attention, forward kernels for __bf16 elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_win_fwd<__bf16>(const Params& p, const FwdPlan& f, hipStream_t s) {
  return launch_fwd_impl<__bf16, true>(p, f, s);
}

}  // namespace attn
}  // namespace ssc
