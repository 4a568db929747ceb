// The gated delta rule's gradients of every chunk, and the limits of its launches.
#include "delta_grad.h"

namespace kda {

bool delta_grad_fits(const DeltaGrad &p) {
  return delta_slots((int64_t)p.B * p.T, p.N, delta_chunk(linear_tile(p.K), p.is_bf16)) * p.H <= most_blocks(512);
}

hipError_t launch_delta_grad(const DeltaGrad &p, hipStream_t st) {
  return p.is_bf16 ? launch_grad_width<bf16_t>(p, st) : launch_grad_width<float>(p, st);
}

}  // namespace kda
