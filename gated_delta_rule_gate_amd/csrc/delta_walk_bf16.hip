// The gated delta rule's forward walk with bf16 inputs.
#include "delta_walk.h"

namespace kda {

hipError_t launch_delta_walk_bf16(const DeltaWalk &p, hipStream_t st) { return launch_delta_width<bf16_t>(p, st); }

}  // namespace kda
