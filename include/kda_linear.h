/*
 * kda_linear.h -- linear attention with one decay per head, on MI355X (gfx950).
 *
 * Per (sequence, head) an FP32 state S in R^{K x V} and, token by token,
 *
 *     S_t = exp(g_t) S_{t-1} + k_t v_t^T
 *     o_t = S_t^T (q_t * scale),        scale = 1/sqrt(K) unless given,
 *
 * as a chunked forward for prompts, its gradient, and the token-sequential
 * recurrence for decoding. It is what KDA becomes without its delta rule and
 * with one decay for all channels of a head, and shares KDA's conventions
 * (kda.h): device pointers only, asynchronous on `stream`, no allocation, no
 * host read of cu_seqlens, caller-owned buffers and workspace, contiguous
 * row-major layouts
 *     q, k [B, T, Hk, K]   v, o [B, T, H, V]   (bf16 or fp32)
 *     g    fp32, natural-log decay, g <= 0: [B, T, H] or [H] (args->decay)
 *     h0, ht [N, H, K, V] fp32        cu_seqlens [N + 1] int32
 * packed batches with B == 1 and N + 1 offsets, rows outside
 * [cu_seqlens[0], cu_seqlens[N]) neither read nor written, an empty slot's
 * final state its h0 bit for bit (zeros without h0), and value head h reading
 * q/k head h / (H / Hk). Statuses and kda_last_error are those of kda.h.
 *   - g = -inf (or any decay under 2^-160) resets the state: nothing before the
 *     token reaches it or any later token.
 *   - State, decays and their sums are held in fp32 or wider. Products run on
 *     the bf16 matrix cores with every fp32 operand taken as a sum of bf16
 *     parts, so fp32 results (states, dg, and every output of fp32 calls)
 *     carry fp32 rounding, not bf16's.
 *   - Outputs must not overlap inputs, other than ht on h0 itself.
 *   - fp32 inputs above 3.38e38 (bf16's largest value) count as infinite.
 *   - A NaN or infinity in q, k or v, or a g that is NaN or +infinity, makes
 *     outputs of its (sequence, head) non-finite, from the start of the 64-token
 *     chunk that holds it (the backward: throughout the sequence), and no other
 *     sequence's or head's, but for sums over them: dq and dk of a shared q/k
 *     head, and dg [H].
 *   - With T == 0 the per-token tensors may be NULL and every final state is
 *     its h0.
 */
#ifndef KDA_LINEAR_H_
#define KDA_LINEAR_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KDA_DECAY_TOKEN = 0, /* g [B, T, H]: a decay for every token and head                     */
  KDA_DECAY_HEAD = 1   /* g [H]: one fixed decay per head (retention layers)                */
} kda_decay_kind;

typedef struct {
  int B, T, H, K, V;     /* sizes as in kda_args; 1 <= H <= 4096                            */
  int N;                 /* sequences (slots); dense: N == B                                */
  int Hk;                /* heads of q and k; 0 means H; H a multiple of it                 */
  kda_dtype dtype;       /* of q, k, v, o (and of d_o, dq, dk, dv)                          */
  kda_decay_kind decay;  /* layout of g and dg                                              */
  float scale;           /* query scale; <= 0 selects 1/sqrt(K)                             */
} kda_linear_args;

/*
 * Bytes of device workspace that kda_linear_chunk_fwd needs (0 when the
 * arguments are invalid or none is needed). Depends on the sizes and on the
 * compute units of the current device: long sequences on few heads are cut
 * into segments that run side by side.
 */
size_t kda_linear_chunk_workspace_bytes(const kda_linear_args *args);

/*
 * Chunked forward. Per chunk of L rows with b_r the chunk-local cumulative
 * decay and S the state at its start:
 *     o_r = scale (e^{b_r} S^T q_r + sum over s <= r of e^{b_r - b_s} (q_r . k_s) v_s)
 *     S'  = e^{b_L} S + sum over s of e^{b_L - b_s} k_s v_s^T
 *   h0, ht     fp32 [N, H, K, V] or NULL; ht may be h0 itself (not overlap it otherwise)
 *   workspace  ws_bytes >= kda_linear_chunk_workspace_bytes(args), 256-byte
 *              aligned; may be NULL when that is 0
 * Supported: K and V multiples of 8 in [8, 256], equal or not. Errors:
 * KDA_ERR_NULL, _SHAPE, _DTYPE, _GATE (unknown decay kind), _ALIGN,
 * _WORKSPACE, _UNSUPPORTED (widths, or more work than one launch takes: about
 * 5.5 million (sequence, head, 128 columns) here and in the gradient, 16.7
 * million in the recurrence; found before anything is launched), _HIP.
 */
kda_status kda_linear_chunk_fwd(const kda_linear_args *args, const void *q, const void *k, const void *v,
                                const float *g, const float *h0, const int32_t *cu_seqlens, void *o, float *ht,
                                void *workspace, size_t ws_bytes, void *stream);

/* Bytes of device workspace that kda_linear_chunk_bwd needs (0 when the arguments are invalid). */
size_t kda_linear_chunk_bwd_workspace_bytes(const kda_linear_args *args);

/*
 * Gradients of L = sum(d_o * o) + sum(dht * ht) for the forward of the same
 * arguments; nothing of the forward needs to be kept.
 *   d_o      [B, T, H, V] dtype args->dtype
 *   dht      fp32 [N, H, K, V] or NULL (zero)
 *   dq, dk   [B, T, Hk, K], summed over the value heads that share a q/k head
 *   dv       [B, T, H, V]
 *   dg       fp32, of g as passed: [B, T, H] or [H]
 *   dh0      fp32 [N, H, K, V] or NULL; an empty slot's is its dht (zeros without dht)
 * No gradient may overlap an input. Results do not depend on the run: every
 * sum has a fixed order.
 */
kda_status kda_linear_chunk_bwd(const kda_linear_args *args, const void *q, const void *k, const void *v,
                                const float *g, const float *h0, const int32_t *cu_seqlens, const void *d_o,
                                const float *dht, void *dq, void *dk, void *dv, float *dg, float *dh0,
                                void *workspace, size_t ws_bytes, void *stream);

/*
 * Token-sequential recurrence, for decoding: one kernel, the fp32 state in
 * registers over a sequence's tokens. Arguments as kda_linear_chunk_fwd,
 * without a workspace. ht may be h0 itself (in-place state update).
 */
kda_status kda_linear_recurrent_fwd(const kda_linear_args *args, const void *q, const void *k, const void *v,
                                    const float *g, const float *h0, const int32_t *cu_seqlens, void *o, float *ht,
                                    void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LINEAR_H_ */
