// The chunk walk of linear attention, fp32 inputs, in token order.
#include "linear_walk.h"

namespace kda {

hipError_t launch_linear_walk_f32_fwd(const LinearWalk &p, hipStream_t st) {
  switch (p.OPL) {
    case 3: return launch_width<float, false, 3>(p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace kda
