// Kernel parameter block and launcher declarations of the query/key norm with
// rotation, shared by its host API and its kernels (qk_norm_rope.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct QkRope {
  const void *q, *k;
  const float *q_weight, *k_weight;
  const int32_t *pos;
  const float *freq;
  void *qo, *ko;               // forward: out; backward: dq, dk (contiguous)
  const void *dqo, *dko;       // backward: gradients of the outputs
  float *part;                 // backward: [blocks][2][D] sums of the weights' gradients, or null
  float *dq_weight, *dk_weight;
  int64_t tokens;
  int64_t qs, ks, qos, kos;    // elements a token
  int H, Hk, D, rot;
  int axes, sec[4];            // sec: spread: limits axes * sections; else ends of the sections
  bool is_bf16, adjacent, spread, normed, l2;
  float eps;
};
hipError_t launch_qk_rope_fwd(const QkRope &p, hipStream_t st);
hipError_t launch_qk_rope_bwd(const QkRope &p, hipStream_t st);
size_t qk_rope_part_bytes(const QkRope &p);

}  // namespace kda
