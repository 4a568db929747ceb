// The gated delta rule's forward walk with fp32 inputs, three bf16 parts each.
#include "delta_walk.h"

namespace kda {

hipError_t launch_delta_walk_f32(const DeltaWalk &p, hipStream_t st) { return launch_delta_width<float>(p, st); }

}  // namespace kda
