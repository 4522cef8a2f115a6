/*
 * rope.h — C ABI of rotary positions on MI355X (gfx950): every token at a position of its
 * own, forward and backward.
 *
 * Pair i (0 <= i < rope_dims / 2) of a head turns by theta_i a position. With
 * theta_i = rope_base^(-2i / rope_dims):
 *
 *   ROPE_SCALING_NONE      theta_i
 *   ROPE_SCALING_LINEAR    theta_i / factor
 *   ROPE_SCALING_BY_PARTS  theta_i (g_i + (1 - g_i) / factor), where
 *                          r_i = original_tokens theta_i / (2 pi), the pair's turns over the
 *                          length that the model was made for, and
 *                          g_i = min(max((r_i - low_turns) / (high_turns - low_turns), 0), 1)
 *
 * (Su et al., "RoFormer: Enhanced Transformer with Rotary Position Embedding", 2021; Chen et
 * al., "Extending Context Window of Large Language Models via Positional Interpolation",
 * 2023; Peng et al., "YaRN: Efficient Context Window Extension of Large Language Models",
 * 2023, whose attention temperature is `magnitude`.) For a token at position p, with (a, b)
 * the pair's elements - i and i + rope_dims / 2 of the head (ROPE_PAIRS_HALF), or 2i and
 * 2i + 1 (ROPE_PAIRS_INTERLEAVED) - and m = magnitude:
 *
 *   a' = m (a cos(p theta_i) - b sin(p theta_i))
 *   b' = m (b cos(p theta_i) + a sin(p theta_i))
 *
 * Elements from rope_dims on, and v, are copied. The backward pass is the transpose: the
 * same with the sines' signs turned. Angles are exact to 2^-31 of a turn at every position: a
 * pair's turns are a 64-bit binary fraction, times the position, of which whole turns drop
 * out. Sines, cosines and products are fp32, each output rounded once to the storage type.
 * NaN and infinities reach their own pair, as the formulas give them in IEEE arithmetic.
 *
 * positions [b, T] (int32, device memory, read by the kernel: a captured call reads their
 * contents at replay) may hold any number, below 0 too; NULL stands for 0 .. T - 1.
 *
 * Memory: the caller owns every device buffer; the plan owns its table of pairs and is only
 * read by calls, so it may be used from several host threads and streams at once. It has to
 * outlive the replays of graphs that captured them. Errors are
 * the FUSED_PROJ_* codes; fused_proj_strerror() describes them.
 */
#ifndef ROPE_H
#define ROPE_H

#include <stddef.h>
#include <stdint.h>

#include "fused_proj.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ROPE_PAIRS_HALF 0
#define ROPE_PAIRS_INTERLEAVED 1

#define ROPE_SCALING_NONE 0
#define ROPE_SCALING_LINEAR 1
#define ROPE_SCALING_BY_PARTS 2

typedef struct rope_desc {
    int32_t dtype;           /* FUSED_PROJ_BF16 | FUSED_PROJ_F32 */
    int32_t qkv_order;       /* FUSED_PROJ_QKV_CONTIGUOUS | FUSED_PROJ_QKV_GROUPED (rope_split*) */
    int64_t batch;           /* b >= 0 sequences */
    int64_t tokens;          /* T >= 1 tokens of each */
    int64_t n_heads;         /* H >= 1 q heads */
    int64_t n_kv_heads;      /* KVH, dividing H; 0 means H */
    int64_t head_dim;        /* hd, a multiple of 8 up to 4096 */
    int64_t rope_dims;       /* rotated width, even, <= hd; 0 means hd */
    int32_t pairs;           /* ROPE_PAIRS_* */
    int32_t scaling;         /* ROPE_SCALING_* */
    double rope_base;        /* > 0, finite */
    double factor;           /* > 0, finite (not used by ROPE_SCALING_NONE) */
    double low_turns;        /* ROPE_SCALING_BY_PARTS: low_turns < high_turns, both finite */
    double high_turns;
    int64_t original_tokens; /* ROPE_SCALING_BY_PARTS: >= 1 */
    double magnitude;        /* finite; 0 means 1 */
} rope_desc;

typedef struct rope_plan *rope_t;

/* Host-only check. FUSED_PROJ_OK, FUSED_PROJ_EINVAL (malformed: sizes, enums, KVH not
 * dividing H, rope_dims odd or above hd, a number outside its range) or
 * FUSED_PROJ_EUNSUPPORTED: hd not a multiple of 8 or above 4096, H + 2 KVH above 2^16, b or T
 * above 2^31 - 1, b T hd of 2^31 or more, or a pair that turns by more than 8 radians a
 * position (a rope_base or factor far below 1). */
int rope_validate(const rope_desc *desc);

/* Validates and puts the table of pairs into the current device's memory (synchronous; the
 * only call that allocates). Errors: as validate, FUSED_PROJ_EINVAL for out == NULL,
 * FUSED_PROJ_EHIP. */
int rope_create(const rope_desc *desc, rope_t *out);

/* Each of the following enqueues one kernel on `stream` (a hipStream_t; NULL = the legacy
 * default stream) and returns; it allocates nothing and never synchronises. Tensors are
 * contiguous, 16-byte aligned (positions 4-byte), on the plan's device. Errors:
 * FUSED_PROJ_EINVAL (a NULL pointer other than positions, another device current),
 * FUSED_PROJ_EALIGN, FUSED_PROJ_EALIAS (an output that overlaps another or an input),
 * FUSED_PROJ_EHIP. */

/* Splits a projected qkv [b, T, (H + 2*KVH)*hd] (columns in qkv_order, as fused_proj.h has
 * them) into q [b*H, T, hd], k and v [b*KVH, T, hd], q and k rotated. */
int rope_split(rope_t plan, const void *qkv, const int32_t *positions, void *q, void *k, void *v, void *stream);

/* Its backward pass: dqkv from dq, dk and dv. */
int rope_split_backward(rope_t plan, const void *dq, const void *dk, const void *dv, const int32_t *positions,
                        void *dqkv, void *stream);

/* Rotates head-major q [b*H, T, hd] and k [b*KVH, T, hd] into q_out and k_out, which may be q
 * and k themselves. */
int rope_rotate(rope_t plan, const void *q, const void *k, const int32_t *positions, void *q_out, void *k_out,
                void *stream);

/* Its backward pass: the gradients of q and k (in place too) from those of q_out and k_out. */
int rope_rotate_backward(rope_t plan, const void *dq_out, const void *dk_out, const int32_t *positions, void *dq,
                         void *dk, void *stream);

/* Frees the plan and its table. NULL is accepted. */
int rope_destroy(rope_t plan);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_H */
