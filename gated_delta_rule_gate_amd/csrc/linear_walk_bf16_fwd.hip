// The chunk walk of linear attention, bf16 inputs, in token order.
#include "linear_walk.h"

namespace kda {

hipError_t launch_linear_walk_bf16_fwd(const LinearWalk &p, hipStream_t st) {
  switch (p.OPL) {
    case 2: return launch_width<bf16_t, false, 2>(p, st);
    case 3: return launch_width<bf16_t, false, 3>(p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace kda
