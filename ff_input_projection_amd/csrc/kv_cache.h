// What the key/value cache's kernels share (the format and the meaning of every size are in
// include/kv_cache.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/kv_cache.h"
#include "fused_proj_kernels.h"

namespace fp {

struct CacheArgs {
    const void* q;             // attend: [b*H, T, hd]
    const void* k;             // write: [b*KVH, T, hd]; read: the same, written
    const void* v;
    uint8_t* k_codes;          // [pages, KVH, page, hd bits / 8]
    uint8_t* v_codes;
    uint32_t* k_params;        // [pages, KVH, page]: scale in the low half, zero in the high
    uint32_t* v_params;
    const int32_t* table;      // [b, max_pages]
    const int32_t* lengths;    // [b]
    const int32_t* counts;     // [b], or nullptr
    void* o;                   // [b, T, H*hd]
    float* part_o;             // attend, split: [splits, rows, hd]
    float* part_ml;            // [splits, rows, 2]
    int64_t page_rows;         // KVH * page_size: rows of a page
    int32_t batch, T, H, KVH, hd, n_pages, max_pages, page_size;
    int32_t capacity;          // max_pages * page_size
    int32_t group;             // H / KVH
    int32_t row_blocks;        // attend: workgroups over a k/v head's query rows
    int32_t splits;            // attend: parts that a sequence's positions are cut into
    float logit_scale;         // sm_scale log2(e)
    int32_t q_limit;           // the exponent field from which on a query's values are too large
    FastDivU31 div_t, div_kvh, div_page, div_group, div_blocks;
};

// A sequence's state as the kernels use it, whatever lengths and counts hold.
struct Step {
    int32_t length;   // positions in the cache, 0..capacity
    int32_t count;    // the step's real tokens, 0..T
    int32_t first;    // position of token 0, perhaps below 0 (or past the capacity)
};
__device__ __forceinline__ Step step_of(const CacheArgs& a, int seq) {
    Step s;
    const int32_t len = max(a.lengths[seq], 0);
    s.count = a.counts ? min(max(a.counts[seq], 0), a.T) : a.T;
    s.first = len - s.count;   // both are 0 or more: no overflow
    s.length = min(len, a.capacity);
    return s;
}

// Defined in kv_attend.hip.
struct AttendPlan {
    bool chunk = false;          // many rows: kv_attend_chunk_kernel
    int32_t row_tiles = 0;       // else: rows of a workgroup, in tiles of 16
    int32_t row_blocks = 0, splits = 0;
    size_t workspace = 0;
};
bool plan_attend(const kv_cache_desc& d, int64_t kvh, AttendPlan* out);   // false: not supported
hipError_t launch_attend(const kv_cache_desc& d, const AttendPlan& p, const CacheArgs& a, hipStream_t st);

}  // namespace fp
