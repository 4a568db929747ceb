// The chunk walk of linear attention, fp32 inputs, in reverse. Three
// bf16 parts hold every fp32 operand.
#include "linear_walk.h"

namespace kda {

hipError_t launch_linear_walk_f32_rev(const LinearWalk &p, hipStream_t st) {
  return p.u ? launch_width<float, true, 3, kDots>(p, st) : launch_width<float, true, 3, kOut>(p, st);
}

}  // namespace kda
