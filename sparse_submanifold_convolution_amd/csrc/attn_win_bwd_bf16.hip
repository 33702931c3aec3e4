// Windowed attention, backward kernels for __bf16 elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_win_bwd<__bf16>(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s) {
  return launch_bwd_impl<__bf16, true>(p, b, w, s);
}

}  // namespace attn
}  // namespace ssc
