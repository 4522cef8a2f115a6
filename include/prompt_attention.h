/*
 * prompt_attention.h — C ABI of attention over whole prompts on MI355X (gfx950), forward and
 * backward: every sequence's tokens attend to the tokens of the same sequence.
 *
 * Query head h = kvh H / KVH + i reads k/v head kvh. Token i sees the tokens j of its sequence,
 * where causal only those with j <= i:
 *
 *   x_ij  = sm_scale sum_d q_i[d] k_j[d]
 *   lse_i = log sum_j exp(x_ij)
 *   o_i   = sum_j exp(x_ij - lse_i) v_j
 *
 * Backward, with p_ij = exp(x_ij - lse_i), D_i = sum_d do_i[d] o_i[d] and
 * ds_ij = p_ij (sum_d do_i[d] v_j[d] - D_i):
 *
 *   dq_i = sm_scale sum_j ds_ij k_j
 *   dk_j = sm_scale sum_i ds_ij q_i     dv_j = sum_i p_ij do_i
 *
 * the last two over all query heads of the k/v head (Vaswani et al., "Attention Is All You
 * Need", 2017; the softmax over tiles with a running maximum and sum: Milakov and Gimelshein,
 * "Online normalizer calculation for softmax", 2018; its gradient from lse and D: Rabe and
 * Staats, "Self-attention Does Not Need O(n^2) Memory", 2021, and Dao et al., 2022).
 *
 * Sequences. sequences = 0: a padded batch; sequence i is the first extents[i] of the T tokens of
 * batch row i (all T where extents is NULL). sequences = n > 0 (batch 1): packed; sequence i is the
 * tokens extents[i] .. extents[i + 1] - 1, extents holding n + 1 ascending offsets; some may be
 * empty, and tokens before the first and behind the last belong to none. extents is device memory, read by
 * the kernels (a captured call reads its contents at replay); numbers outside 0 .. T count as the
 * nearer bound, and offsets that do not ascend cut the tokens between the first and the last
 * offset at each of them. Tokens of no sequence get zeros in o, dq, dk and dv and -infinity in
 * lse, and nothing of theirs reaches another token.
 *
 * Numerics. Products of bf16 numbers are exact, their sums, the softmax and its statistics fp32; the
 * probabilities are rounded to bf16 for their products with v and do, ds to the sum of two bf16
 * numbers for those with k and q; each output is rounded once. D_i is summed as p_ij dp_ij, not from
 * the rounded o, for dk, and for the dq_i of tokens that see at most 128. Logits are fp32: x_ij log2(e) stays below 2^127. A NaN or an
 * infinity reaches the tokens that the formulas lead it to, and no token that does not see it.
 * Results do not depend on timing: no atomics in global memory.
 *
 * Errors are the FUSED_PROJ_* codes; fused_proj_strerror() describes them. A plan only holds
 * sizes, so it may be used from several host threads and streams at once.
 */
#ifndef PROMPT_ATTENTION_H
#define PROMPT_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "fused_proj.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct prompt_attention_desc {
    int32_t dtype;        /* FUSED_PROJ_BF16 (the only type supported) */
    int32_t causal;       /* 1: a token sees itself and earlier ones; 0: its whole sequence */
    int64_t batch;        /* b >= 0 */
    int64_t tokens;       /* T >= 1 tokens of a batch row */
    int64_t n_heads;      /* H >= 1 query heads */
    int64_t n_kv_heads;   /* KVH, dividing H; 0 means H */
    int64_t head_dim;     /* hd, a multiple of 8 up to 256 */
    int64_t sequences;    /* 0: padded; n > 0: packed, batch 1 */
    int64_t q_strides[3]; /* elements between batch rows, heads and tokens of q, k and v; a head's */
    int64_t k_strides[3]; /* elements are next to each other. Multiples of 8, >= 0. The head-major */
    int64_t v_strides[3]; /* outputs of fused_proj.h: heads T hd, T hd, hd */
    double sm_scale;      /* > 0; sm_scale log2(e) between 2^-126 and 2^128; 0 means 1 / sqrt(hd) */
} prompt_attention_desc;

typedef struct prompt_attention_plan *prompt_attention_t;

/* Host-only check. FUSED_PROJ_OK, FUSED_PROJ_EINVAL (malformed: sizes, flags, KVH not dividing H,
 * strides below 0, packed sequences with another batch than 1, sm_scale outside its range) or
 * FUSED_PROJ_EUNSUPPORTED: not bf16, hd no multiple of 8 or above 256, strides no multiples
 * of 8, a token stride above 2^24, T of 2^30 or more, sequences of 2^30 or more, b T H of
 * 2^31 or more, b H at or above 2^23 / ceil(T / 64) rounded down, or an address beyond 2^60. */
int prompt_attention_validate(const prompt_attention_desc *desc);

/* Validates and fixes the split of the work; touches no GPU memory. Errors: as validate,
 * FUSED_PROJ_EINVAL for out == NULL, FUSED_PROJ_EHIP. */
int prompt_attention_create(const prompt_attention_desc *desc, prompt_attention_t *out);

/* Enqueues the forward pass on `stream` (a hipStream_t; NULL = the legacy default stream) and
 * returns; allocates nothing, never synchronises.
 *   q, k, v   device, laid out as the descriptor says, 16-byte aligned
 *   extents   device int32 [b] or [sequences + 1]; may be NULL where sequences is 0
 *   o         device [b, T, H*hd] (token-major: what a projection of it reads), 16-byte aligned
 *   lse       device fp32 [b*H, T] (natural logarithms); NULL where no backward pass wants it
 * Errors: FUSED_PROJ_EINVAL (a NULL pointer, another device current), FUSED_PROJ_EALIGN,
 * FUSED_PROJ_EALIAS (an output overlapping another or an input), FUSED_PROJ_EHIP. */
int prompt_attention_run(prompt_attention_t plan, const void *q, const void *k, const void *v, const int32_t *extents,
                         void *o, void *lse, void *stream);

/* Bytes of device workspace prompt_attention_backward needs (0 when there are no tokens). */
int prompt_attention_backward_workspace_size(prompt_attention_t plan, size_t *bytes);

/* Enqueues the backward pass. q, k, v, extents: the forward pass's; o, lse: its outputs; d_o: the
 * upstream gradient [b, T, H*hd]; dq [b, H, T, hd], dk and dv [b, KVH, T, hd]: head-major and
 * dense whatever the inputs' strides. workspace: device, at least the size above, 16-byte
 * aligned; its contents do not matter, and calls that share it must not overlap in time.
 * Errors as prompt_attention_run; a short workspace is FUSED_PROJ_EINVAL. */
int prompt_attention_backward(prompt_attention_t plan, const void *q, const void *k, const void *v,
                              const int32_t *extents, const void *o, const void *lse, const void *d_o, void *dq,
                              void *dk, void *dv, void *workspace, size_t workspace_bytes, void *stream);

/* Frees the plan. NULL is accepted. */
int prompt_attention_destroy(prompt_attention_t plan);

#ifdef __cplusplus
}
#endif

#endif /* PROMPT_ATTENTION_H */
