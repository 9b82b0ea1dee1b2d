// The reversed sweeps of linear attention (gradients of keys and values): the
// instantiations of linattn_sweep.h that run from the last token to the first.
#include "linattn_sweep.h"

namespace linattn {

hipError_t launch_reverse(const SweepPlan& p, hipStream_t s) {
  return p.a.K <= 64 ? launch_types<64, true>(p, s) : launch_types<128, true>(p, s);
}

}  // namespace linattn
