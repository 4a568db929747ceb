// The chunk walk of linear attention, bf16 inputs, in reverse. Scores and
// state enter a bf16 y as two bf16 parts (what they leave out, 2^-16, is far
// below y's own rounding; one part would add as much error again as that
// rounding), and as three where the rows' dots are summed over many tokens.
#include "linear_walk.h"

namespace kda {

hipError_t launch_linear_walk_bf16_rev(const LinearWalk &p, hipStream_t st) {
  return p.u ? launch_width<bf16_t, true, 3, kDots>(p, st) : launch_width<bf16_t, true, 2, kOut>(p, st);
}

}  // namespace kda
