// The key/value cache in 4 or 8 bits: quantising a step's k and v into their slots and
// reading slots back as values (gfx950; the format is in include/kv_cache.h), and the C ABI
// of the cache and of the attention over it (kv_attend.hip).
//
// Both move bytes (2 hd + hd bits / 8 + 4 a row): a row is LPR neighbouring lanes, each with
// 8 values, 16 bytes of the bf16 side and 4 or 8 of the cache's. The least and greatest
// value of a row are found across its lanes, so k and v are read once and nothing is kept
// in LDS. Measured, 98304 rows of 64 in 8 bits, three quarters of them real: write 9 us
// (35 MB, 3.9 TB/s), read 8 us (34 MB, 4.3 TB/s); 256 rows of 128 in 4 bits: 3 us each, a
// launch's own time.
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
    if (s >= st.count) return -1;
    const int32_t p = st.first + s;
    if (p < 0 || p >= a.capacity) return -1;
    const int32_t pg = (int32_t)fp::fastdiv_u31((uint32_t)p, a.div_page);
    const int32_t page = a.table[(int64_t)seq * a.max_pages + pg];
    if (page < 0 || page >= a.n_pages) return -1;
    return (int64_t)page * a.page_rows + (int64_t)head * a.page_size + (p - pg * a.page_size);
}

// The least of v over groups of LPR lanes (LPR a power of two); NaN where there is one.
template <int LPR>
__device__ __forceinline__ float group_min(float v) {
    const auto least = [](float a, float b) { return __builtin_elementwise_minimum(a, b); };
    if constexpr (LPR > 1) v = least(v, dpp<kQuadXor1>(v));
    if constexpr (LPR > 2) v = least(v, dpp<kQuadXor2>(v));
    if constexpr (LPR > 4) v = least(v, dpp<kHalfMirror>(v));   // quads hold one value each
    if constexpr (LPR > 8) v = least(v, dpp<kRowRor8>(v));
    if constexpr (LPR > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = least(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if constexpr (LPR > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = least(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}

struct RowAt {
    int64_t in;     // row of k and of v
    int64_t slot;   // row of the cache, or -1
    int piece;      // the lane's 8 values
    bool lane;      // whether it has any
};
// Row and piece of this thread: 256 / LPR rows of k and of v a workgroup. Both of a token
// lie in the same slot, so a thread takes both: one search for the slot, two loads in flight.
template <int LPR>
__device__ __forceinline__ RowAt row_at(const CacheArgs& a) {
    RowAt r;
    const int64_t rows = (int64_t)a.batch * a.KVH * a.T;
    r.in = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    r.lane = r.in < rows;
    if (!r.lane) r.in = 0;
    const uint32_t slab = fp::fastdiv_u31((uint32_t)r.in, a.div_t), seq = fp::fastdiv_u31(slab, a.div_kvh);
    r.slot = slot_of(a, (int)seq, (int)(slab - seq * (uint32_t)a.KVH), (int)((uint32_t)r.in - slab * (uint32_t)a.T));
    r.piece = threadIdx.x % LPR;
    return r;
}

template <int BITS>
struct Codes;   // 8 of them
template <>
struct Codes<4> {
    uint32_t w;
    __device__ __forceinline__ void set(int e, uint32_t c) { w = e ? w | c << (4 * e) : c; }
    __device__ __forceinline__ float get(int e) const { return (float)((w >> (4 * e)) & 15u); }
};
template <>
struct Codes<8> {
    u32x2 w;
    __device__ __forceinline__ void set(int e, uint32_t c) { w[e >> 2] = e & 3 ? w[e >> 2] | c << (8 * (e & 3)) : c; }
    __device__ __forceinline__ float get(int e) const { return (float)((w[e >> 2] >> (8 * (e & 3))) & 255u); }
};

// A row's codes and params from its values, 8 in this lane.
template <int BITS, int LPR>
__device__ __forceinline__ void quantise(const u32x4& h, Codes<BITS>& codes, uint32_t& params) {
    constexpr float kMost = (float)((1 << BITS) - 1);
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
    const float scale = __uint_as_float((__float_as_uint((high - low) / kMost) + 0xFFFFu) & 0xFFFF0000u);
    const bool ok = scale <= 0x1p24f;   // not so for NaN
    // (x - zero) / scale as IEEE division rounds it, with one division a row: where inv is 1 /
    // scale correctly rounded and q within a step of the quotient, q + (d - q scale) inv rounds
    // to the quotient (Markstein, "Computation of elementary functions on the IBM RISC
    // System/6000 processor", 1990). The remainder is exact while nothing underflows; rows of
    // smaller scales divide.
    const float inv = 1.0f / scale;
    float quotient[8];
    if (scale >= 0x1p-80f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = f[e] - low, q = d * inv;
            quotient[e] = fmaf(fmaf(-q, scale, d), inv, q);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) quotient[e] = (f[e] - low) / scale;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        // 0 / 0 where scale is 0, and every value of a row kept as NaN: 0
        codes.set(e, ok && scale > 0.0f ? (uint32_t)fminf(rintf(quotient[e]), kMost) : 0u);
    params = ok ? (__float_as_uint(scale) >> 16) | (__float_as_uint(low) & 0xFFFF0000u) : 0x7FC07FC0u;
}

template <int BITS, int LPR>
__global__ __launch_bounds__(256) void kv_cache_write_kernel(CacheArgs a) {
    const RowAt r = row_at<LPR>(a);
    const int pieces = a.hd >> 3;
    // lanes past the row's end take its first piece: it changes neither bound
    const int64_t at = r.in * a.hd + (r.piece < pieces ? r.piece : 0) * 8;
    const u32x4 k = *reinterpret_cast<const u32x4*>(static_cast<const __bf16*>(a.k) + at);
    const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const __bf16*>(a.v) + at);
    Codes<BITS> kc, vc;
    uint32_t kp, vp;
    quantise<BITS, LPR>(k, kc, kp);
    quantise<BITS, LPR>(v, vc, vp);
    if (!r.lane || r.slot < 0) return;
    if (r.piece < pieces) {
        reinterpret_cast<Codes<BITS>*>(a.k_codes)[r.slot * pieces + r.piece] = kc;
        reinterpret_cast<Codes<BITS>*>(a.v_codes)[r.slot * pieces + r.piece] = vc;
    }
    if (r.piece == 0) {
        a.k_params[r.slot] = kp;
        a.v_params[r.slot] = vp;
    }
}

// The lane's 8 values; scale code is exact (8 + bits significant bits), so one rounding to fp32.
template <int BITS>
__device__ __forceinline__ u32x4 values(const Codes<BITS>& c, uint32_t params) {
    const float scale = __uint_as_float(params << 16), zero = __uint_as_float(params & 0xFFFF0000u);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = fmaf(scale, c.get(e), zero);
    return Piece<__bf16>::pack(f);
}

template <int BITS, int LPR>
__global__ __launch_bounds__(256) void kv_cache_read_kernel(CacheArgs a) {
    const RowAt r = row_at<LPR>(a);
    const int pieces = a.hd >> 3;
    if (!r.lane || r.piece >= pieces) return;
    u32x4 k = {0, 0, 0, 0}, v = k;
    if (r.slot >= 0) {
        const Codes<BITS> kc = reinterpret_cast<const Codes<BITS>*>(a.k_codes)[r.slot * pieces + r.piece];
        const Codes<BITS> vc = reinterpret_cast<const Codes<BITS>*>(a.v_codes)[r.slot * pieces + r.piece];
        const uint32_t kp = a.k_params[r.slot], vp = a.v_params[r.slot];
        k = values<BITS>(kc, kp);
        v = values<BITS>(vc, vp);
    }
    const int64_t at = r.in * a.hd + r.piece * 8;
    *reinterpret_cast<u32x4*>(static_cast<__bf16*>(const_cast<void*>(a.k)) + at) = k;
    *reinterpret_cast<u32x4*>(static_cast<__bf16*>(const_cast<void*>(a.v)) + at) = v;
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

// Logits are in units of log 2.
float logits_factor(const kv_cache_desc& d) {
    const double scale = d.sm_scale > 0.0 ? d.sm_scale : 1.0 / std::sqrt((double)d.head_dim);
    return (float)(scale * 1.4426950408889634074);
}

int check(const kv_cache_desc* d, Derived* out) {
    if (!d) return FUSED_PROJ_EINVAL;
    if (d->dtype != FUSED_PROJ_BF16 && d->dtype != FUSED_PROJ_F32) return FUSED_PROJ_EINVAL;
    if (d->bits != 4 && d->bits != 8) return FUSED_PROJ_EINVAL;
    if (d->batch < 0 || d->tokens < 1 || d->n_heads < 1 || d->head_dim < 1 || d->n_kv_heads < 0) return FUSED_PROJ_EINVAL;
    if (d->n_kv_heads > 0 && d->n_heads % d->n_kv_heads != 0) return FUSED_PROJ_EINVAL;
    if (d->page_size < 1 || d->n_pages < 1 || d->max_pages < 1) return FUSED_PROJ_EINVAL;
    if (!(d->sm_scale >= 0.0) || !std::isfinite(logits_factor(*d))) return FUSED_PROJ_EINVAL;
    if (d->dtype != FUSED_PROJ_BF16) return FUSED_PROJ_EUNSUPPORTED;
    if (d->head_dim % 8 != 0 || d->head_dim > 512) return FUSED_PROJ_EUNSUPPORTED;
    if (d->page_size % 16 != 0 || d->page_size > 65536) return FUSED_PROJ_EUNSUPPORTED;
    if (d->n_pages > kMaxIndex || d->max_pages > kMaxIndex || d->max_pages * d->page_size > kMaxIndex / 2)
        return FUSED_PROJ_EUNSUPPORTED;
    Derived r;
    r.kvh = d->n_kv_heads > 0 ? d->n_kv_heads : d->n_heads;
    r.q_rows = mul_cap(mul_cap(d->batch, d->tokens), d->n_heads);
    if (d->n_heads > kMaxIndex || d->tokens > kMaxIndex || d->batch > kMaxIndex || r.q_rows < 0 || r.q_rows > kMaxIndex)
        return FUSED_PROJ_EUNSUPPORTED;
    if (mul_cap(d->n_heads, d->tokens) > kMaxIndex / 2 || mul_cap(d->batch, d->max_pages) < 0) return FUSED_PROJ_EUNSUPPORTED;
    r.rows = d->batch * r.kvh * d->tokens;
    const int64_t slots = mul_cap(mul_cap(d->n_pages, r.kvh), d->page_size);
    r.codes = mul_cap(slots, d->head_dim * d->bits / 8);
    r.params = mul_cap(slots, 4);
    if (slots < 0 || r.codes < 0 || r.params < 0) return FUSED_PROJ_EUNSUPPORTED;
    r.lpr = 1;
    while (r.lpr * 8 < d->head_dim) r.lpr *= 2;
    if (r.rows * r.lpr > kMaxIndex) return FUSED_PROJ_EUNSUPPORTED;   // threads of one grid
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
    const unsigned grid = (unsigned)((r.rows * r.lpr + 255) / 256);
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
    a.logit_scale = logits_factor(h->d);
    // 2^90, or less where the logits' factor is 2^7 or more: see lift_of in kv_attend.hip
    const int e = a.logit_scale > 0.0f ? std::ilogb(a.logit_scale) : 0;
    a.q_limit = 127 + 90 - (e > 6 ? e - 6 : 0);
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
