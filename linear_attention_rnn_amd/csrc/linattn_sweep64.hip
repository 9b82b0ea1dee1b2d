// The sweeps of linear attention with up to 64 key channels.
#include "linattn_sweep.h"

namespace linattn {

hipError_t launch_sweeps64(const SweepPlan& p, hipStream_t s) { return launch_types<64>(p, s); }

}  // namespace linattn
