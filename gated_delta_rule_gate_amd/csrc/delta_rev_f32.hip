// The gated delta rule's gradient walk with fp32 inputs, three bf16 parts each.
#include "delta_rev.h"

namespace kda {

hipError_t launch_delta_rev_f32(const DeltaWalk &p, hipStream_t st) { return launch_rev_width<float>(p, st); }

}  // namespace kda
