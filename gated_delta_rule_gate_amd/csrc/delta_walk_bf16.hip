// The gated delta rule's forward walk with bf16 inputs.
#include "delta_walk.h"

namespace kda {

// A bf16 o takes two parts of the state and the scores: with one, their own
// rounding would add to o's.
hipError_t launch_delta_walk_bf16(const DeltaWalk &p, hipStream_t st) { return launch_delta_width<bf16_t, 2>(p, st); }

}  // namespace kda
