// The key/value cache in 4 or 8 bits: quantising a step's k and v into their slots and
// reading slots back as values (gfx950; the format is in include/kv_cache.h), and the C ABI
// of the cache and of the attention over it (kv_attend.hip).
//
// Both move bytes (2 hd + hd bits / 8 + 4 a row, and 15 VALU operations a value for the
// IEEE division where the memory rate allows 60): a row is LPR neighbouring lanes, each with
// 8 values, 16 bytes of the bf16 side and 4 or 8 of the cache's. The least and greatest
// value of a row are found across its lanes, so k and v are read once and nothing is kept
// in LDS.
#include <cmath>
#include <cstring>
#include <new>

#include "kv_cache.h"
#include "vector_io.h"

namespace {

using namespace fp::dev;
using fp::CacheArgs;

// Where a row of the step lies in the cache: its row index, or -1 for none.
__device__ __forceinline__ int64_t slot_of(const CacheArgs& a, int seq, int head, int s) {
    const fp::Step st = fp::step_of(a, seq);
    const int32_t p = st.first + s;
    if (s >= st.count || p < 0 || p >= a.capacity) return -1;
    const int32_t pg = (int32_t)fp::fastdiv_u31((uint32_t)p, a.div_page);
    const int32_t page = a.table[(int64_t)seq * a.max_pages + pg];
    if (page < 0 || page >= a.n_pages) return -1;
    return (int64_t)page * a.page_rows + (int64_t)head * a.page_size + (p - pg * a.page_size);
}

// The least of v over groups of LPR lanes (LPR a power of two); NaN where there is one.
template <int LPR>
__device__ __forceinline__ float group_min(float v) {
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) v = __builtin_elementwise_minimum(v, __shfl_xor(v, m));
    return v;
}

struct RowAt {
    int64_t in;     // row of k or v
    int64_t slot;   // row of the cache, or -1
    int piece;      // the lane's 8 values
    bool lane;      // whether it has any
    bool value;     // v rather than k
};
// Row and piece of this thread: 256 / LPR rows a workgroup, k's rows first.
template <int LPR>
__device__ __forceinline__ RowAt row_at(const CacheArgs& a) {
    RowAt r;
    const int64_t rows = (int64_t)a.batch * a.KVH * a.T;
    int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    r.lane = row < 2 * rows;
    if (!r.lane) row = 0;
    r.value = row >= rows;
    r.in = r.value ? row - rows : row;
    const uint32_t slab = fp::fastdiv_u31((uint32_t)r.in, a.div_t), seq = fp::fastdiv_u31(slab, a.div_kvh);
    r.slot = slot_of(a, (int)seq, (int)(slab - seq * (uint32_t)a.KVH), (int)((uint32_t)r.in - slab * (uint32_t)a.T));
    r.piece = threadIdx.x % LPR;
    return r;
}

template <int BITS, int LPR>
__global__ __launch_bounds__(256) void kv_cache_write_kernel(CacheArgs a) {
    constexpr float kMost = (float)((1 << BITS) - 1);
    const RowAt r = row_at<LPR>(a);
    const int pieces = a.hd >> 3;
    // lanes past the row's end take its first piece: it changes neither bound
    const __bf16* x = static_cast<const __bf16*>(r.value ? a.v : a.k) + r.in * a.hd + (r.piece < pieces ? r.piece : 0) * 8;
    const u32x4 h = *reinterpret_cast<const u32x4*>(x);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = Piece<__bf16>::get(h, e);
    float low = f[0], high = -f[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        low = __builtin_elementwise_minimum(low, f[e]);
        high = __builtin_elementwise_minimum(high, -f[e]);
    }
    low = group_min<LPR>(low);
    high = -group_min<LPR>(high);
    // up to the next bfloat16 number: the bits of a number >= 0 are ordered as it is
    float scale = __uint_as_float((__float_as_uint((high - low) / kMost) + 0xFFFFu) & 0xFFFF0000u);
    const bool ok = scale <= 0x1p24f;   // not so for NaN
    uint32_t code[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float c = rintf((f[e] - low) / scale);
        // 0 / 0 where scale is 0, and every value of a row kept as NaN: 0
        code[e] = ok && scale > 0.0f ? (uint32_t)fminf(c, kMost) : 0u;
    }
    if (!r.lane || r.slot < 0) return;
    uint8_t* codes = r.value ? a.v_codes : a.k_codes;
    if (r.piece < pieces) {
        if constexpr (BITS == 4) {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) w |= code[e] << (4 * e);
            *reinterpret_cast<uint32_t*>(codes + (r.slot * pieces + r.piece) * 4) = w;
        } else {
            u32x2 w = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e >> 2] |= code[e] << (8 * (e & 3));
            *reinterpret_cast<u32x2*>(codes + (r.slot * pieces + r.piece) * 8) = w;
        }
    }
    if (r.piece == 0) {
        uint32_t* params = r.value ? a.v_params : a.k_params;
        params[r.slot] = ok ? (__float_as_uint(scale) >> 16) | (__float_as_uint(low) & 0xFFFF0000u) : 0x7FC07FC0u;
    }
}

template <int BITS, int LPR>
__global__ __launch_bounds__(256) void kv_cache_read_kernel(CacheArgs a) {
    const RowAt r = row_at<LPR>(a);
    const int pieces = a.hd >> 3;
    if (!r.lane || r.piece >= pieces) return;
    float f[8];
    if (r.slot < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.0f;
    } else {
        const uint8_t* codes = r.value ? a.v_codes : a.k_codes;
        const uint32_t w = (r.value ? a.v_params : a.k_params)[r.slot];
        const float scale = __uint_as_float(w << 16), zero = __uint_as_float(w & 0xFFFF0000u);
        // scale code is exact (8 + bits significant bits), so one rounding to fp32
        if constexpr (BITS == 4) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + (r.slot * pieces + r.piece) * 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(scale, (float)((c >> (4 * e)) & 15u), zero);
        } else {
            const u32x2 c = *reinterpret_cast<const u32x2*>(codes + (r.slot * pieces + r.piece) * 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(scale, (float)((c[e >> 2] >> (8 * (e & 3))) & 255u), zero);
        }
    }
    __bf16* x = static_cast<__bf16*>(const_cast<void*>(r.value ? a.v : a.k)) + r.in * a.hd + r.piece * 8;
    *reinterpret_cast<u32x4*>(x) = Piece<__bf16>::pack(f);
}

// ------------------------------------------------------------------ plans
constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;

int64_t mul_cap(int64_t a, int64_t b) {
    const int64_t lim = int64_t(1) << 60;
    if (a < 0 || b < 0) return -1;
    if (a == 0 || b == 0) return 0;
    return a > lim / b ? -1 : a * b;
}

struct Derived {
    int64_t kvh = 0, rows = 0, q_rows = 0, codes = 0, params = 0;   // rows of k; bytes of the storage
    int lpr = 0;
};

int check(const kv_cache_desc* d, Derived* out) {
    if (!d) return FUSED_PROJ_EINVAL;
    if (d->dtype != FUSED_PROJ_BF16 && d->dtype != FUSED_PROJ_F32) return FUSED_PROJ_EINVAL;
    if (d->bits != 4 && d->bits != 8) return FUSED_PROJ_EINVAL;
    if (d->batch < 0 || d->tokens < 1 || d->n_heads < 1 || d->head_dim < 1 || d->n_kv_heads < 0) return FUSED_PROJ_EINVAL;
    if (d->n_kv_heads > 0 && d->n_heads % d->n_kv_heads != 0) return FUSED_PROJ_EINVAL;
    if (d->page_size < 1 || d->n_pages < 1 || d->max_pages < 1) return FUSED_PROJ_EINVAL;
    if (!(d->sm_scale >= 0.0) || !std::isfinite((float)d->sm_scale)) return FUSED_PROJ_EINVAL;
    if (d->dtype != FUSED_PROJ_BF16) return FUSED_PROJ_EUNSUPPORTED;
    if (d->head_dim % 8 != 0 || d->head_dim > 512) return FUSED_PROJ_EUNSUPPORTED;
    if (d->page_size % 16 != 0 || d->page_size > 65536) return FUSED_PROJ_EUNSUPPORTED;
    if (d->n_pages > kMaxIndex || d->max_pages > kMaxIndex || d->max_pages * d->page_size > kMaxIndex)
        return FUSED_PROJ_EUNSUPPORTED;
    Derived r;
    r.kvh = d->n_kv_heads > 0 ? d->n_kv_heads : d->n_heads;
    r.q_rows = mul_cap(mul_cap(d->batch, d->tokens), d->n_heads);
    if (d->n_heads > kMaxIndex || d->tokens > kMaxIndex || d->batch > kMaxIndex || r.q_rows < 0 || r.q_rows > kMaxIndex)
        return FUSED_PROJ_EUNSUPPORTED;
    if (mul_cap(d->n_heads, d->tokens) > kMaxIndex || mul_cap(d->batch, d->max_pages) < 0) return FUSED_PROJ_EUNSUPPORTED;
    r.rows = d->batch * r.kvh * d->tokens;
    const int64_t slots = mul_cap(mul_cap(d->n_pages, r.kvh), d->page_size);
    r.codes = mul_cap(slots, d->head_dim * d->bits / 8);
    r.params = mul_cap(slots, 4);
    if (slots < 0 || r.codes < 0 || r.params < 0) return FUSED_PROJ_EUNSUPPORTED;
    r.lpr = 1;
    while (r.lpr * 8 < d->head_dim) r.lpr *= 2;
    if (out) *out = r;
    return FUSED_PROJ_OK;
}

struct Range {
    uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes}; }
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }
bool misaligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1); }

int hip_status(hipError_t e) {
    if (e == hipSuccess) return FUSED_PROJ_OK;
    fp::set_last_hip_error(e);
    return FUSED_PROJ_EHIP;
}

}  // namespace

struct kv_cache_plan {
    kv_cache_desc d;
    Derived r;
    fp::AttendPlan attend;
    bool can_attend = false;
    int device = -1;
};

namespace {

// The checks that every call shares, and its arguments. `wide` are the call's own 16-byte
// aligned buffers, the first `n_out` of them outputs; the storage is an output when writing.
int prepare(const kv_cache_plan* h, const kv_cache_storage* s, const int32_t* table, const int32_t* lengths,
            const int32_t* counts, const Range* wide, int n_wide, int n_out, bool writes, CacheArgs* out) {
    const kv_cache_desc& d = h->d;
    const Derived& r = h->r;
    if (!s || !s->k_codes || !s->k_params || !s->v_codes || !s->v_params || !table || !lengths) return FUSED_PROJ_EINVAL;
    for (int i = 0; i < n_wide; ++i)
        if (!wide[i].lo) return FUSED_PROJ_EINVAL;
    for (int i = 0; i < n_wide; ++i)
        if (wide[i].lo & 15u) return FUSED_PROJ_EALIGN;
    for (const void* p : {s->k_codes, s->k_params, s->v_codes, s->v_params})
        if (misaligned(p, 16)) return FUSED_PROJ_EALIGN;
    for (const void* p : {(const void*)table, (const void*)lengths, (const void*)counts})
        if (misaligned(p, 4)) return FUSED_PROJ_EALIGN;
    Range outs[8], ins[16];
    int no = 0, ni = 0;
    for (int i = 0; i < n_wide; ++i) (i < n_out ? outs[no++] : ins[ni++]) = wide[i];
    const Range store[4] = {range(s->k_codes, r.codes), range(s->k_params, r.params), range(s->v_codes, r.codes),
                            range(s->v_params, r.params)};
    for (const Range& x : store) (writes ? outs[no++] : ins[ni++]) = x;
    ins[ni++] = range(table, d.batch * d.max_pages * 4);
    ins[ni++] = range(lengths, d.batch * 4);
    ins[ni++] = range(counts, counts ? d.batch * 4 : 0);
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return FUSED_PROJ_EALIAS;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return FUSED_PROJ_EALIAS;
    }
    int dev = -1;
    const int rc = hip_status(hipGetDevice(&dev));
    if (rc) return rc;
    if (dev != h->device) return FUSED_PROJ_EINVAL;
    CacheArgs a;
    std::memset(&a, 0, sizeof(a));
    a.k_codes = static_cast<uint8_t*>(s->k_codes);
    a.v_codes = static_cast<uint8_t*>(s->v_codes);
    a.k_params = static_cast<uint32_t*>(s->k_params);
    a.v_params = static_cast<uint32_t*>(s->v_params);
    a.table = table;
    a.lengths = lengths;
    a.counts = counts;
    a.page_rows = r.kvh * d.page_size;
    a.batch = (int32_t)d.batch;
    a.T = (int32_t)d.tokens;
    a.H = (int32_t)d.n_heads;
    a.KVH = (int32_t)r.kvh;
    a.hd = (int32_t)d.head_dim;
    a.n_pages = (int32_t)d.n_pages;
    a.max_pages = (int32_t)d.max_pages;
    a.page_size = (int32_t)d.page_size;
    a.capacity = (int32_t)(d.max_pages * d.page_size);
    a.group = (int32_t)(d.n_heads / r.kvh);
    a.div_t = fp::make_fastdiv_u31((uint32_t)a.T);
    a.div_kvh = fp::make_fastdiv_u31((uint32_t)a.KVH);
    a.div_page = fp::make_fastdiv_u31((uint32_t)a.page_size);
    a.div_group = fp::make_fastdiv_u31((uint32_t)a.group);
    *out = a;
    return FUSED_PROJ_OK;
}

template <int BITS>
void launch_rows(const Derived& r, const CacheArgs& a, bool write, hipStream_t st) {
    const unsigned grid = (unsigned)((2 * r.rows * r.lpr + 255) / 256);
#define KV_CASE(L)                                                                                     \
    if (r.lpr == L) {                                                                                  \
        if (write)                                                                                     \
            hipLaunchKernelGGL((kv_cache_write_kernel<BITS, L>), dim3(grid), dim3(256), 0, st, a);     \
        else                                                                                           \
            hipLaunchKernelGGL((kv_cache_read_kernel<BITS, L>), dim3(grid), dim3(256), 0, st, a);      \
        return;                                                                                        \
    }
    KV_CASE(1) KV_CASE(2) KV_CASE(4) KV_CASE(8) KV_CASE(16) KV_CASE(32) KV_CASE(64)
#undef KV_CASE
}

int run_rows(const kv_cache_plan* h, CacheArgs a, const void* k, const void* v, bool write, void* stream) {
    a.k = k;
    a.v = v;
    if (h->d.bits == 4)
        launch_rows<4>(h->r, a, write, static_cast<hipStream_t>(stream));
    else
        launch_rows<8>(h->r, a, write, static_cast<hipStream_t>(stream));
    return hip_status(hipGetLastError());
}

}  // namespace

extern "C" {

int kv_cache_validate(const kv_cache_desc* desc) { return check(desc, nullptr); }

int kv_cache_create(const kv_cache_desc* desc, kv_cache_t* out) {
    if (!out) return FUSED_PROJ_EINVAL;
    *out = nullptr;
    Derived r;
    int rc = check(desc, &r);
    if (rc) return rc;
    kv_cache_plan* h = new (std::nothrow) kv_cache_plan();
    if (!h) return FUSED_PROJ_EHIP;
    h->d = *desc;
    h->r = r;
    h->can_attend = fp::plan_attend(*desc, r.kvh, &h->attend);
    rc = hip_status(hipGetDevice(&h->device));
    if (rc) {
        delete h;
        return rc;
    }
    *out = h;
    return FUSED_PROJ_OK;
}

int kv_cache_storage_bytes(kv_cache_t h, size_t* codes, size_t* params) {
    if (!h || !codes || !params) return FUSED_PROJ_EINVAL;
    *codes = (size_t)h->r.codes;
    *params = (size_t)h->r.params;
    return FUSED_PROJ_OK;
}

int kv_cache_write(kv_cache_t h, const void* k, const void* v, const kv_cache_storage* storage, const int32_t* table,
                   const int32_t* lengths, const int32_t* counts, void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (h->r.rows == 0) return FUSED_PROJ_OK;
    const int64_t bytes = h->r.rows * h->d.head_dim * 2;
    const Range wide[2] = {range(k, bytes), range(v, bytes)};
    CacheArgs a;
    const int rc = prepare(h, storage, table, lengths, counts, wide, 2, 0, true, &a);
    return rc ? rc : run_rows(h, a, k, v, true, stream);
}

int kv_cache_read(kv_cache_t h, const kv_cache_storage* storage, const int32_t* table, const int32_t* lengths,
                  const int32_t* counts, void* k, void* v, void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (h->r.rows == 0) return FUSED_PROJ_OK;
    const int64_t bytes = h->r.rows * h->d.head_dim * 2;
    const Range wide[2] = {range(k, bytes), range(v, bytes)};
    CacheArgs a;
    const int rc = prepare(h, storage, table, lengths, counts, wide, 2, 2, false, &a);
    return rc ? rc : run_rows(h, a, k, v, false, stream);
}

int kv_cache_attend_workspace_size(kv_cache_t h, size_t* bytes) {
    if (!h || !bytes) return FUSED_PROJ_EINVAL;
    if (!h->can_attend) return FUSED_PROJ_EUNSUPPORTED;
    *bytes = h->attend.workspace;
    return FUSED_PROJ_OK;
}

int kv_cache_attend(kv_cache_t h, const void* q, const kv_cache_storage* storage, const int32_t* table,
                    const int32_t* lengths, const int32_t* counts, void* o, void* workspace, size_t workspace_bytes,
                    void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (!h->can_attend) return FUSED_PROJ_EUNSUPPORTED;
    if (h->r.q_rows == 0) return FUSED_PROJ_OK;
    const size_t need = h->attend.workspace;
    if (need > 0 && (!workspace || workspace_bytes < need)) return FUSED_PROJ_EINVAL;
    const int64_t bytes = h->r.q_rows * h->d.head_dim * 2;
    Range wide[3] = {range(o, bytes), range(workspace, (int64_t)need), range(q, bytes)};
    if (need == 0) {
        wide[1] = wide[2];
    }
    CacheArgs a;
    int rc = prepare(h, storage, table, lengths, counts, wide, need ? 3 : 2, need ? 2 : 1, false, &a);
    if (rc) return rc;
    a.q = q;
    a.o = o;
    a.row_blocks = h->attend.row_blocks;
    a.splits = h->attend.splits;
    a.div_blocks = fp::make_fastdiv_u31((uint32_t)a.row_blocks);
    const double scale = h->d.sm_scale > 0.0 ? h->d.sm_scale : 1.0 / std::sqrt((double)h->d.head_dim);
    a.logit_scale = (float)(scale * 1.4426950408889634074);
    if (need) {
        a.part_o = static_cast<float*>(workspace);
        a.part_ml = a.part_o + (int64_t)a.splits * h->r.q_rows * h->d.head_dim;
    }
    return hip_status(fp::launch_attend(h->d, h->attend, a, static_cast<hipStream_t>(stream)));
}

int kv_cache_destroy(kv_cache_t h) {
    delete h;
    return FUSED_PROJ_OK;
}

}  // extern "C"
