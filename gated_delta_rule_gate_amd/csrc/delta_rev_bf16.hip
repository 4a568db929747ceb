// The gated delta rule's gradient walk with bf16 inputs.
#include "delta_rev.h"

namespace kda {

hipError_t launch_delta_rev_bf16(const DeltaWalk &p, hipStream_t st) { return launch_rev_width<bf16_t>(p, st); }

}  // namespace kda
