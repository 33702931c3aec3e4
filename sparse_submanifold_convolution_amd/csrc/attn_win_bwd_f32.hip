// Windowed attention, backward kernels for float elements.
#include "attn.h"

namespace ssc {
namespace attn {

template <>
int launch_win_bwd<float>(Params p, const BwdPlan& b, const BwdParts& w, hipStream_t s) {
  return launch_bwd_impl<float, true>(p, b, w, s);
}

}  // namespace attn
}  // namespace ssc
