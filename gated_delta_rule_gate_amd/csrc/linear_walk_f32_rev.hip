// The chunk walk of linear attention, fp32 inputs, in reverse.
#include "linear_walk.h"

namespace kda {

hipError_t launch_linear_walk_f32_rev(const LinearWalk &p, hipStream_t st) {
  switch (p.OPL) {
    case 3: return launch_width<float, true, 3>(p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace kda
