/*
 * layer_norm.h — C ABI of the MI355X (gfx950) layer norm that feeds the fused input
 * projection, and of its backward pass.
 *
 * For every token t of a channels-first [b, c, spatial...] or token-major [b, s, c]
 * activation (the layouts of fused_proj.h, read where they lie):
 *
 *   mean[t] = sum_c x[t, c] / C
 *   rstd[t] = 1 / sqrt(sum_c (x[t, c] - mean[t])^2 / C + eps)
 *   y[t, c] = (x[t, c] - mean[t]) rstd[t] gamma[c] + beta[c]
 *
 * (Ba, Kiros and Hinton, "Layer Normalization", 2016). Backward, with
 * xhat = (x - mean) rstd and g = dy gamma:
 *
 *   dx[t, c]  = rstd[t] (g[t, c] - sum_c g / C - xhat[t, c] sum_c (g xhat) / C)
 *   dgamma[c] = sum_t dy[t, c] xhat[t, c]
 *   dbeta[c]  = sum_t dy[t, c]
 *
 * Sums, statistics and every intermediate value are fp32 (the last stage of dgamma and
 * dbeta is a 64-bit sum); each output is rounded once to the storage type. Results do not
 * depend on timing: no atomics. NaN and infinities reach their own token's y and dx, and
 * their channel's dgamma and dbeta, as the formulas give them. Sums beyond fp32's range are
 * infinite: with a value 2^64 away from the mean the variance is, and rstd 0.
 *
 * Memory: the caller owns every device buffer. Errors are the FUSED_PROJ_* codes;
 * fused_proj_strerror() describes them. A plan only holds sizes, so it may be used from
 * several host threads and streams at once.
 */
#ifndef LAYER_NORM_H
#define LAYER_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "fused_proj.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct layer_norm_desc {
    int32_t dtype;            /* FUSED_PROJ_BF16 | FUSED_PROJ_F32: x, gamma, beta and every gradient */
    int32_t x_layout;         /* FUSED_PROJ_X_* */
    int64_t batch;            /* b >= 0 */
    int64_t channels;         /* C >= 1 */
    int32_t n_spatial;        /* 1..3 for channels-first, exactly 1 for tokens-last */
    int64_t spatial[3];       /* S = their product, >= 0 */
    int64_t x_stride_batch;   /* element strides of x, all >= 0, any alignment */
    int64_t x_stride_channel;
    int64_t x_stride_spatial[3];
    int32_t has_bias;         /* 1: beta[C] is added, and has a gradient */
    double eps;               /* >= 0, finite */
} layer_norm_desc;

typedef struct layer_norm_plan *layer_norm_t;

/* Host-only check. FUSED_PROJ_OK, FUSED_PROJ_EINVAL (malformed: sizes, enums, strides or
 * eps below 0) or FUSED_PROJ_EUNSUPPORTED: channels-first spatial strides that do not
 * flatten into one unit-stride token index, a tokens-last x_stride_channel other than 1
 * (either only where that stride is ever used), tokens-last C above 32768, or b*S, S, C or
 * b*S*C beyond 2^31 - 2^23, the same, 2^29 or 2^60. Any C and S, odd ones too. */
int layer_norm_validate(const layer_norm_desc *desc);

/* Validates and picks the kernels; touches no GPU memory. Errors: as validate,
 * FUSED_PROJ_EINVAL for out == NULL, FUSED_PROJ_EHIP. */
int layer_norm_create(const layer_norm_desc *desc, layer_norm_t *out);

/* Enqueues the forward pass on `stream` (a hipStream_t; NULL = the legacy default stream)
 * and returns; one kernel, allocates nothing, never synchronises.
 *   x      device, laid out as the descriptor says
 *   gamma  device [C]; beta device [C] when has_bias, else ignored
 *   y      device, dense in x's logical shape ([b, C, S] or [b, S, C])
 *   stats  device fp32 [2, b*S]: the means, then the rstds; NULL when not wanted
 * Errors: FUSED_PROJ_EINVAL (NULL pointer, another device current), FUSED_PROJ_EALIGN (a
 * pointer not aligned to its element), FUSED_PROJ_EALIAS (y or stats overlapping each other or an
 * input), FUSED_PROJ_EHIP. */
int layer_norm_run(layer_norm_t plan, const void *x, const void *gamma, const void *beta, void *y, void *stats,
                   void *stream);

/* Bytes of device workspace layer_norm_backward needs (0 when there are no tokens). */
int layer_norm_backward_workspace_size(layer_norm_t plan, size_t *bytes);

/* Enqueues the backward pass on `stream` (asynchronous; two kernels, no allocation).
 *   x, gamma  the forward inputs; stats the forward's fp32 [2, b*S]
 *   dy        device, dense in x's logical shape
 *   dx        device, dense in x's logical shape; dgamma, dbeta device [C] (dbeta only
 *             when has_bias)
 *   workspace device, layer_norm_backward_workspace_size bytes; contents do not matter.
 *             Calls that share a workspace must not overlap in time.
 * With no tokens dgamma and dbeta are set to zero. Errors as layer_norm_run; a short
 * workspace is FUSED_PROJ_EINVAL, one not 16-byte aligned FUSED_PROJ_EALIGN. */
int layer_norm_backward(layer_norm_t plan, const void *x, const void *gamma, const void *stats, const void *dy,
                        void *dx, void *dgamma, void *dbeta, void *workspace, size_t workspace_bytes, void *stream);

/* Frees the plan. NULL is accepted. */
int layer_norm_destroy(layer_norm_t plan);

#ifdef __cplusplus
}
#endif

#endif /* LAYER_NORM_H */
