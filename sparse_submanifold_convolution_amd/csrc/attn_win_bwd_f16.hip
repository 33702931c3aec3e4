// Windowed attention, backward kernels for _Float16 elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_win_bwd<_Float16>(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s) {
  return launch_bwd_impl<_Float16, true>(p, b, w, s);
}

}  // namespace attn
}  // namespace ssc
