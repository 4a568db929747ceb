/*
 * kda_rope.h -- the norm of every head's query and key row and their rotation
 * by position, in one pass, on MI355X (gfx950).
 *
 * Per row x of D channels (one token and head), with the tensor's own weight:
 *
 *     n = weight x / sqrt(mean(x^2) + eps)       (norm RMS; L2: sum in place of mean; or none)
 *     y = n with its first `rot` channels turned, pair by pair:
 *         (y_a, y_b) = (n_a cos t - n_b sin t, n_b cos t + n_a sin t),
 *         t = position inv_freq[i], pair i = channels (i, i + rot/2), or (2i, 2i + 1)
 *
 * with positions on one to four axes (time, height and width of images and
 * video), every frequency i reading one of them. Angles and their reduction to
 * an eighth of a turn and less are fp64 (three roundings: an angle of 2^31 is off
 * by less than 2^-22 turns), their sines and cosines fp32, within 2^-23, norms,
 * products and weights' gradients fp32 or wider; y is rounded once. It makes
 * the q and k rows of the attention operators: with norm L2 and rot 0 the l2
 * norm that kda_chunk_fwd and kda_delta_chunk_fwd expect. Conventions as in kda.h: device
 * pointers, asynchronous on `stream`, no allocation.
 */
#ifndef KDA_ROPE_H_
#define KDA_ROPE_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { KDA_QK_RMS = 0, KDA_QK_L2 = 1, KDA_QK_NONE = 2 } kda_qk_norm_kind;
typedef enum { KDA_PAIRS_HALF = 0, KDA_PAIRS_ADJACENT = 1 } kda_pair_layout;

typedef struct {
  int64_t tokens;          /* B T, >= 0                                                           */
  int H, Hk, D;            /* heads of q and of k, >= 1; D a multiple of 8 in [8, 512]            */
  int rot;                 /* channels turned: a multiple of 8 in [0, D]; 0: no rotation          */
  kda_dtype dtype;         /* of q and k (and their gradients)                                    */
  kda_qk_norm_kind norm;
  kda_pair_layout pairs;
  int axes;                /* axes of the positions, 1 to 4                                       */
  int sections[4];         /* with axes > 1: frequencies of each axis, summing to rot / 2         */
  int spread;              /* 0: an axis' frequencies are neighbours, in the axes' order; 1: axis
                              a >= 1 takes frequencies a, a + axes, a + 2 axes, ... (sections[a]
                              of them, below rot / 2), axis 0 all others                          */
  float eps;               /* >= 0; with 0 a row of zeros has no norm: its results are NaN        */
  int64_t q_stride, k_stride;    /* elements from a token's rows to the next's of q and k (of a
                              fused projection): multiples of 8, at least the heads' H D or Hk D; 0: that */
  int64_t qo_stride, ko_stride;  /* the same of the outputs (in the backward: of the outputs' gradients) */
} kda_qk_args;

/*
 *   q [tokens, H, D], k [tokens, Hk, D]     q_weight, k_weight  fp32 [D] or NULL (ones)
 *   positions  int32 [axes, tokens]         inv_freq  fp32 [rot / 2]    (both NULL with rot 0)
 *   q_out, k_out   as q and k; each may be its input itself, at the same stride
 * Errors: KDA_ERR_NULL, _SHAPE (sizes, strides, sections), _DTYPE, _GATE
 * (unknown norm or pair layout), _ALIGN, _UNSUPPORTED (D, rot), _HIP.
 */
kda_status kda_qk_norm_rope_fwd(const kda_qk_args *args, const void *q, const void *k, const float *q_weight,
                                const float *k_weight, const int32_t *positions, const float *inv_freq,
                                void *q_out, void *k_out, void *stream);

/* Bytes of device workspace that kda_qk_norm_rope_bwd needs (0 when the arguments are invalid). */
size_t kda_qk_norm_rope_bwd_workspace_bytes(const kda_qk_args *args);

/*
 * Gradients of sum(dq_out * q_out) + sum(dk_out * k_out) for the forward of the same arguments.
 *   dq [tokens, H, D], dk [tokens, Hk, D]   contiguous; either may be its dq_out or dk_out itself
 *                                           where that is contiguous
 *   dq_weight, dk_weight   fp32 [D] or NULL (not wanted)
 *   workspace   ws_bytes >= kda_qk_norm_rope_bwd_workspace_bytes(args), 256-byte aligned;
 *               may be NULL when no weight's gradient is wanted
 * Every sum over rows has a fixed order.
 */
kda_status kda_qk_norm_rope_bwd(const kda_qk_args *args, const void *q, const void *k, const float *q_weight,
                                const float *k_weight, const int32_t *positions, const float *inv_freq,
                                const void *dq_out, const void *dk_out, void *dq, void *dk, float *dq_weight,
                                float *dk_weight, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ROPE_H_ */
