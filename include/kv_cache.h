/*
 * kv_cache.h — C ABI of the MI355X (gfx950) key/value cache in 4 or 8 bits that takes the
 * k and v of a fused projection (or a split + RoPE), and of the attention over it.
 *
 * A step has up to T tokens in each of b sequences. After it the cache holds lengths[i]
 * tokens of sequence i; the last counts[i] of them (0 <= counts[i] <= T; T where counts is
 * NULL) are the step's own: token s < counts[i] of the step is at position
 * lengths[i] - counts[i] + s of the sequence. Tokens s >= counts[i] are padding.
 * Rotations are the caller's: a projection's or a split + RoPE's plan rotates from one
 * pos_offset, so sequences at different positions take a plan each.
 *
 * Format. A row is the hd values x of one token of one k/v head, in k or in v:
 *
 *   zero  = min x                                  (bfloat16, as x is)
 *   scale = the least bfloat16 number >= (max x - zero) / (2^bits - 1)
 *   code  = min(rint((x - zero) / scale), 2^bits - 1), ties to even; 0 where scale is 0
 *
 * and stands for zero + scale code. x - zero, the quotients and their rounding are IEEE
 * fp32 operations. Asymmetric uniform quantisation by rows; the scale is rounded up so that
 * the largest value keeps the largest code. A row that holds a NaN or an infinity, or whose
 * scale would exceed 2^24, is kept as scale = zero = NaN: it reads back as NaN, never as
 * wrong finite values.
 *
 * Storage (the caller's device memory; the same for every plan with the same n_kv_heads,
 * head_dim, bits, page_size and n_pages, whatever its batch and tokens):
 *   k_codes, v_codes    bytes [n_pages, KVH, page_size, hd bits / 8]; with 4 bits element
 *                       2i is the low half of byte i, element 2i + 1 the high half
 *   k_params, v_params  bfloat16 [n_pages, KVH, page_size, 2]: scale, zero
 * table [b, max_pages] (int32): position p of sequence i is slot p % page_size of page
 * table[i, p / page_size]. An entry outside 0 .. n_pages - 1 is no page: nothing is written
 * there, it reads as zeros, and attention does not see its positions. The same holds for
 * positions at or past max_pages page_size. lengths below 0 count as 0, counts outside
 * 0 .. T as the nearer bound, and a token at a position below 0 as padding. table, lengths
 * and counts are device memory, read by the kernels: no call waits for them, and a captured
 * call reads their contents at replay.
 *
 * Attention. Query head h = kvh H / KVH + i reads k/v head kvh. For token s < counts[i] at
 * position p, with khat and vhat what the rows stand for:
 *
 *   x[j] = sm_scale sum_d q[d] khat[j, d]             positions j <= p
 *   o    = sum_j exp(x[j] - max x) vhat[j] / sum_j exp(x[j] - max x)
 *
 * and 0 for a padding token, or where no position is seen. Products of q and codes are
 * exact, sums, softmax and statistics fp32, the probabilities (times v's scale) rounded to
 * bfloat16 for the second product, o rounded once. Rows of v may hold numbers of any size;
 * besides its roundings o is off by up to about 2^-90, where products with codes vanish. A
 * query row that holds a NaN, an infinity or a value of 2^90 or more (2^96 divided by the
 * greatest power of two in sm_scale log2(e), where that is less) gives NaN where it sees any
 * position; so does every row that sees a row kept as NaN. Logits are fp32: with x[j] log2(e)
 * of 2^127 or more a row's output is not defined. Positions that a token does not see never
 * reach its output, whatever their slots hold. Nor do other queries, but that those of one
 * workgroup share a power of two, whose rounding is at most 2^-39 of a key's scale in a logit.
 * Softmax over tiles with a running maximum and sum: Milakov and Gimelshein, "Online normalizer
 * calculation for softmax", 2018.
 *
 * Errors are the FUSED_PROJ_* codes; fused_proj_strerror() describes them. A plan only holds
 * sizes, so it may be used from several host threads and streams at once. Calls that write
 * and calls that use the same slots must be ordered by the caller (the same stream does).
 */
#ifndef KV_CACHE_H
#define KV_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "fused_proj.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kv_cache_desc {
    int32_t dtype;       /* FUSED_PROJ_BF16 (the only type supported): q, k, v and o */
    int32_t bits;        /* 4 | 8 */
    int64_t batch;       /* b >= 0 sequences */
    int64_t tokens;      /* T >= 1 tokens of a step, the padded length */
    int64_t n_heads;     /* H >= 1 query heads */
    int64_t n_kv_heads;  /* KVH, dividing H; 0 means H */
    int64_t head_dim;    /* hd, a multiple of 8 up to 512; attention: 32, 64, 96, 128, 192 or 256 */
    int64_t page_size;   /* positions of a page, a multiple of 16 up to 65536 */
    int64_t n_pages;     /* pages of the storage, >= 1 */
    int64_t max_pages;   /* pages of a sequence (the table's width), >= 1 */
    double sm_scale;     /* > 0, sm_scale log2(e) below 2^128; 0 means 1 / sqrt(hd) */
} kv_cache_desc;

typedef struct kv_cache_plan *kv_cache_t;

/* The cache's memory. */
typedef struct kv_cache_storage {
    void *k_codes, *k_params, *v_codes, *v_params;
} kv_cache_storage;

/* Host-only check. FUSED_PROJ_OK, FUSED_PROJ_EINVAL (malformed: sizes, enums, KVH not
 * dividing H, sm_scale outside its range) or FUSED_PROJ_EUNSUPPORTED (not bf16,
 * head_dim or page_size outside the ranges above, max_pages page_size or T H of 2^30 or
 * more, b T H or b T KVH times head_dim / 8 (rounded up to a power of two) of 2^31 or more,
 * storage of 2^60 bytes or more). */
int kv_cache_validate(const kv_cache_desc *desc);

/* Validates and fixes the split of the work; touches no GPU memory. Errors: as validate,
 * FUSED_PROJ_EINVAL for out == NULL, FUSED_PROJ_EHIP. */
int kv_cache_create(const kv_cache_desc *desc, kv_cache_t *out);

/* Bytes of k_codes (and of v_codes), and of k_params (and of v_params). */
int kv_cache_storage_bytes(kv_cache_t plan, size_t *codes, size_t *params);

/* Enqueues the quantisation of the step's k and v ([b*KVH, T, hd], as fused_proj_run and
 * split_rope_run write them) into their slots on `stream` (a hipStream_t; NULL = the legacy
 * default stream); one kernel, allocates nothing, never synchronises. Slots that are not the
 * step's are left as they were. No slot may be two tokens' in one call (its contents would
 * be either's, or a mixture). Every pointer is 16-byte aligned, table, lengths and counts
 * 4-byte (FUSED_PROJ_EALIGN); storage may not overlap itself or an input
 * (FUSED_PROJ_EALIAS); FUSED_PROJ_EINVAL: a NULL pointer (but counts), or another device
 * current; FUSED_PROJ_EHIP: a failed launch. */
int kv_cache_write(kv_cache_t plan, const void *k, const void *v, const kv_cache_storage *storage,
                   const int32_t *table, const int32_t *lengths, const int32_t *counts, void *stream);

/* Enqueues the reverse: the step's rows of the cache as values into k and v [b*KVH, T, hd],
 * zeros for padding and absent pages. With counts = lengths (T the longest) that is all the
 * cache holds, from position 0. Errors as kv_cache_write. */
int kv_cache_read(kv_cache_t plan, const kv_cache_storage *storage, const int32_t *table, const int32_t *lengths,
                  const int32_t *counts, void *k, void *v, void *stream);

/* Bytes of device workspace kv_cache_attend needs for this plan (0 if none). */
int kv_cache_attend_workspace_size(kv_cache_t plan, size_t *bytes);

/* Enqueues the attention of the step's queries q [b*H, T, hd] (as fused_proj_run writes
 * them) over the cache into o [b, T, H*hd] (token-major: what a projection of the attention's
 * output reads). The step's own k and v are in the cache already. workspace: device, at
 * least kv_cache_attend_workspace_size bytes, contents do not matter; calls that share it
 * must not overlap in time. Errors as kv_cache_write, and FUSED_PROJ_EUNSUPPORTED for a
 * head_dim that attention does not take (or 2^23 workgroups or more), FUSED_PROJ_EINVAL for
 * a short workspace. */
int kv_cache_attend(kv_cache_t plan, const void *q, const kv_cache_storage *storage, const int32_t *table,
                    const int32_t *lengths, const int32_t *counts, void *o, void *workspace, size_t workspace_bytes,
                    void *stream);

/* Frees the plan. NULL is accepted. */
int kv_cache_destroy(kv_cache_t plan);

#ifdef __cplusplus
}
#endif

#endif /* KV_CACHE_H */
