/*
 * kda_norm.h -- the norms round an attention block, fused with its gate and
 * residual branch, on MI355X (gfx950).
 *
 * Per row of D values, with x the block's output:
 *
 *     n = weight x / sqrt(mean(x^2) + eps)       (norm RMS; L2: sum in place of mean)
 *     y = residual + scale n act(gate)           (act: sigmoid or SiLU)
 *     z = next_weight y / sqrt(mean(y^2) + eps)  (the norm before the next block)
 *
 * Every part but the first norm is optional. Rows of a head (D = V, rows =
 * B T H) give the output norm of an attention layer; norm L2 without weight
 * is the l2 norm that kda_chunk_fwd expects of its q and k rows; D = model
 * width with residual and z is a block's whole epilogue.
 * Conventions as in kda.h: contiguous device pointers, 16-byte aligned,
 * asynchronous on `stream`, no allocation. Statistics, products and parameter
 * gradients are fp32 or wider; y and z are each rounded once (z comes from the
 * unrounded y).
 */
#ifndef KDA_NORM_H_
#define KDA_NORM_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { KDA_NORM_RMS = 0, KDA_NORM_L2 = 1 } kda_norm_kind;
typedef enum { KDA_ACT_SIGMOID = 0, KDA_ACT_SILU = 1 } kda_gate_act;

typedef struct {
  int64_t rows;           /* >= 0                                                            */
  int D;                  /* row width: a multiple of 8 in [8, 16384]                        */
  kda_dtype dtype;        /* of x, gate and z (and their gradients)                          */
  kda_dtype res_dtype;    /* of residual and y: dtype or KDA_F32; dtype without a residual   */
  kda_norm_kind norm;     /* of the first norm; the second is always RMS                     */
  kda_gate_act gate_act;  /* of gate, where given                                            */
  float scale;            /* residual scale where scale_vec is NULL                          */
  float eps;              /* >= 0; with 0 a row of zeros has no norm: its results are NaN     */
} kda_norm_args;

/*
 *   x            [rows, D]              weight       fp32 [D] or NULL (ones)
 *   gate         [rows, D] or NULL      residual     [rows, D] (res_dtype) or NULL
 *   scale_vec    fp32 [D] or NULL (args->scale)
 *   next_weight  fp32 [D] or NULL (ones where z is given)
 *   y            [rows, D], res_dtype; may be the residual itself (in place)
 *   z            [rows, D] or NULL (no second norm)
 * Errors: KDA_ERR_NULL, _SHAPE, _DTYPE, _GATE (unknown norm or activation),
 * _ALIGN, _UNSUPPORTED (D), _HIP.
 */
kda_status kda_block_norm_fwd(const kda_norm_args *args, const void *x, const float *weight, const void *gate,
                              const void *residual, const float *scale_vec, const float *next_weight, void *y,
                              void *z, void *stream);

/* Bytes of device workspace that kda_block_norm_bwd needs (0 when the arguments are invalid). */
size_t kda_block_norm_bwd_workspace_bytes(const kda_norm_args *args);

/*
 * Gradients of sum(dy * y) + sum(dz * z) for the forward of the same arguments.
 *   dy          [rows, D], res_dtype, or NULL (zero; only with dz)
 *   dz          [rows, D] or NULL (z was not written, or has no gradient)
 *   dx          [rows, D]
 *   dgate       [rows, D], with gate; dresidual [rows, D] (res_dtype), or NULL.
 *               dresidual may be dy itself
 *   dweight, dscale_vec, dnext_weight   fp32 [D] or NULL (not wanted); dnext_weight needs dz
 *   workspace   ws_bytes >= kda_block_norm_bwd_workspace_bytes(args), 256-byte aligned
 * Every sum over rows has a fixed order.
 */
kda_status kda_block_norm_bwd(const kda_norm_args *args, const void *x, const float *weight, const void *gate,
                              const void *residual, const float *scale_vec, const float *next_weight,
                              const void *dy, const void *dz, void *dx, void *dgate, void *dresidual,
                              float *dweight, float *dscale_vec, float *dnext_weight, void *workspace,
                              size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_NORM_H_ */
