// The sweeps of linear attention with up to 128 key channels.
#include "linattn_sweep.h"

namespace linattn {

hipError_t launch_sweeps128(const SweepPlan& p, hipStream_t s) { return launch_types<128>(p, s); }

}  // namespace linattn
