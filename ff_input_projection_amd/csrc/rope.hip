// Rotary positions (gfx950; formulas and layouts are in include/rope.h).
//
// The op moves bytes: every element is read once and written once. A thread holds one unit
// of a head's row - W pairs and with them 2 W elements, W the widest power of two up to 16
// bytes that divides the halves, or the V elements of a 16-byte piece of an interleaved row -
// computes its sines and cosines once and applies them to G heads of its token, whose
// loads are all under way together. Both elements of a pair are in one thread, so a rotation
// in place needs no order between threads.
//
// Angles. A pair's turns a position are a 64-bit binary fraction f (of which whole turns were
// dropped: positions are whole numbers); p f modulo 2^64 is the angle, exact up to p 2^-64 of
// a turn, by two 32-bit multiplications. Its top 32 bits go to the nearest quarter turn
// and a rest of at most an eighth of a turn, whose sine and cosine are Taylor's series (to
// x^9 and x^10: off by less than 2e-9).
//
// Measured: 2 x 4096 tokens, 96 heads of 128, 403 MB in 82 us, 4.9 TB/s (a large copy: 5.2). Halves that 8 elements (4 of
// fp32) do not divide are moved in smaller accesses: 2 x 4096 tokens, 96 heads of 80, 252 MB, all of a head rotated 71 us, 20 of
// its elements 109, 22 of them 100.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/rope.h"
#include "fused_proj_kernels.h"
#include "vector_io.h"

namespace {

using namespace fp::dev;

// Heads of a thread: 4 share their sines and cosines (2: 2 x 4096 x 96 heads of 128 no faster, 8: a tenth slower), 1 where
// workgroups of 4 would not fill the card (2 x 1024 x 24 heads of 32: 5.7 -> 4.9 us).
constexpr int kHeads = 4;
constexpr int64_t kFewBlocks = 512;
constexpr int64_t kMostDims = 4096;
constexpr long double kTwoPi = 6.283185307179586476925286766559005768L;
// Angles are extended-precision numbers, off by 2^-63 of themselves: up to this many radians a
// position they are exact to 2^-31 of a turn at position 2^31.
constexpr long double kMostAngle = 8.0L;

// One side of the copy: where q, k and v heads lie.
struct Side {
    char* part[3];        // q, k, v
    int32_t token_major;  // 1: all in rows of `width` elements a token; 0: [b*heads, T, hd] each
};
struct RopeArgs {
    Side from, to;
    const int32_t* positions;   // [b, T] or nullptr
    const uint64_t* turns;      // [rd / 2] binary fractions
    int64_t width;              // (H + 2 KVH) hd
    uint32_t items;             // b T units_per_row
    int32_t T, H, KVH, hd, rd, heads;   // heads: H + 2 KVH, or H + KVH where v is not moved
    int32_t units;              // of a head's row
    int32_t grouped, backward;
    float magnitude;
    fp::FastDivU31 div_units, div_t;
};

__device__ __forceinline__ char* row_of(const Side& s, const RopeArgs& a, int head, uint32_t bi, uint32_t t, int esize) {
    const int which = head < a.H ? 0 : head < a.H + a.KVH ? 1 : 2;
    const int h = which == 0 ? head : which == 1 ? head - a.H : head - a.H - a.KVH;
    if (!s.token_major) {
        const int64_t heads = which == 0 ? a.H : a.KVH;
        return s.part[which] + ((((int64_t)bi * heads + h) * a.T + t) * a.hd) * esize;
    }
    int col = head;
    if (a.grouped) {
        const int g = a.H / a.KVH;
        col = which == 0 ? h / g * (g + 2) + h % g : h * (g + 2) + g + which - 1;
    }
    return s.part[0] + (((int64_t)bi * a.T + t) * a.width + (int64_t)col * a.hd) * esize;
}

// cos and sin of `turn` / 2^32 of a turn.
__device__ __forceinline__ void cos_sin(uint32_t turn, float& c, float& s) {
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(turn - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
    const float x2 = x * x;
    float ps = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
    ps = fmaf(ps, x2, 8.3333333e-3f);
    ps = fmaf(ps, x2, -1.6666667e-1f);
    ps = fmaf(ps * x2, x, x);
    float pc = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
    pc = fmaf(pc, x2, -1.3888889e-3f);
    pc = fmaf(pc, x2, 4.1666667e-2f);
    pc = fmaf(pc, x2, -0.5f);
    pc = fmaf(pc, x2, 1.0f);
    const float a = (quarter & 1) ? ps : pc, b = (quarter & 1) ? pc : ps;
    c = __uint_as_float(__float_as_uint(a) ^ (((quarter + 1) & 2) << 30));
    s = __uint_as_float(__float_as_uint(b) ^ ((quarter & 2) << 30));
}
__device__ __forceinline__ uint32_t turn_of(uint64_t f, int32_t p) {
    // bits 32..63 of p f, p taken modulo 2^64
    const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32);
    return __umulhi((uint32_t)p, lo) + (uint32_t)p * hi - (p < 0 ? lo : 0u);
}

template <typename T, int N>
struct alignas(sizeof(T) * N) Unit {
    T x[N];
};

// Past the caches, as nothing is read again here (2 x 4096 x 96 heads of 128: 94 -> 82 us). Attention reads q, k and v next; the two
// together, through the caches / past them: 2 x 4096 tokens, 32 heads on 8 of 128, 348 / 346 us; 1 x 512, 19.0 / 19.5; 512 x 32, 12 of
// 64, 54 / 58; a decoding step of 16 sequences with its cache's write and attention 16.9 / 17.2.
template <typename T, int N>
__device__ __forceinline__ void store_unit(T* p, const Unit<T, N>& u) {
    if constexpr (sizeof(u) == 16)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, u), reinterpret_cast<u32x4*>(p));
    else
        *reinterpret_cast<Unit<T, N>*>(p) = u;
}

// HALF: a unit is W pairs, elements i .. i + W - 1 and i + rd/2 ..; behind the rotated width W
// elements that are copied. Otherwise it is W consecutive elements, pairs inside.
template <typename T, int W, bool HALF, int G>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    if (item >= a.items) return;
    const uint32_t row = fp::fastdiv_u31(item, a.div_units);
    const int unit = (int)(item - row * (uint32_t)a.units);
    const uint32_t bi = fp::fastdiv_u31(row, a.div_t), t = row - bi * (uint32_t)a.T;
    const int half = a.rd >> 1;
    constexpr int P = HALF ? W : W / 2;   // pairs of a unit
    const int pair0 = unit * P;
    // HALF: a unit is rotated or copied whole (W divides half); interleaved: pair by pair
    const bool turns = pair0 < half;
    const int at = HALF && !turns ? a.rd + (pair0 - half) : HALF ? pair0 : pair0 * 2;
    const int head0 = blockIdx.y * G;

    Unit<T, W> x[G], y[G];
#pragma unroll
    for (int g = 0; g < G; ++g)
        if (head0 + g < a.heads) {
            const T* p = reinterpret_cast<const T*>(row_of(a.from, a, head0 + g, bi, t, sizeof(T))) + at;
            x[g] = *reinterpret_cast<const Unit<T, W>*>(p);
            if (HALF && turns) y[g] = *reinterpret_cast<const Unit<T, W>*>(p + half);
        }
    float c[P], s[P];
    if (turns) {
        const int32_t pos = a.positions ? a.positions[row] : (int32_t)t;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const bool in = HALF || pair0 + i < half;
            cos_sin(turn_of(a.turns[in ? pair0 + i : 0], pos), c[i], s[i]);
            c[i] *= a.magnitude;
            s[i] *= a.backward ? -a.magnitude : a.magnitude;
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if (head0 + g >= a.heads) break;
        T* p = reinterpret_cast<T*>(row_of(a.to, a, head0 + g, bi, t, sizeof(T))) + at;
        const bool rotate = turns && head0 + g < a.H + a.KVH;
        if (rotate) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                T& first = HALF ? x[g].x[i] : x[g].x[2 * i];
                T& second = HALF ? y[g].x[i] : x[g].x[2 * i + 1];
                const float u = (float)first, v = (float)second;
                if (HALF || pair0 + i < half) {
                    first = (T)(u * c[i] - v * s[i]);
                    second = (T)(v * c[i] + u * s[i]);
                }
            }
        }
        store_unit(p, x[g]);
        if (HALF && turns) store_unit(p + half, y[g]);
    }
}

// The angle of pair i a position.
long double pair_angle(const rope_desc& d, int64_t rd, int64_t i) {
    const long double theta = powl((long double)d.rope_base, -2.0L * (long double)i / (long double)rd);
    if (d.scaling == ROPE_SCALING_LINEAR) return theta / (long double)d.factor;
    if (d.scaling == ROPE_SCALING_BY_PARTS) {
        const long double r = (long double)d.original_tokens * theta / kTwoPi;
        long double g = (r - d.low_turns) / ((long double)d.high_turns - d.low_turns);
        g = g < 0.0L ? 0.0L : g > 1.0L ? 1.0L : g;
        return theta * (g + (1.0L - g) / (long double)d.factor);
    }
    return theta;
}

struct Derived {
    int64_t kvh = 0, rd = 0, rows = 0;
    int width = 0;   // W
    int units = 0;   // of a head's row
};

bool ok_number(double x) { return std::isfinite(x); }

int check(const rope_desc* d, Derived* out) {
    if (!d) return FUSED_PROJ_EINVAL;
    if (d->dtype != FUSED_PROJ_BF16 && d->dtype != FUSED_PROJ_F32) return FUSED_PROJ_EINVAL;
    if (d->batch < 0 || d->tokens < 1 || d->n_heads < 1 || d->head_dim < 1) return FUSED_PROJ_EINVAL;
    if (d->n_kv_heads < 0 || (d->n_kv_heads > 0 && d->n_heads % d->n_kv_heads != 0)) return FUSED_PROJ_EINVAL;
    if (d->qkv_order != FUSED_PROJ_QKV_CONTIGUOUS && d->qkv_order != FUSED_PROJ_QKV_GROUPED) return FUSED_PROJ_EINVAL;
    if (d->pairs != ROPE_PAIRS_HALF && d->pairs != ROPE_PAIRS_INTERLEAVED) return FUSED_PROJ_EINVAL;
    if (d->scaling < ROPE_SCALING_NONE || d->scaling > ROPE_SCALING_BY_PARTS) return FUSED_PROJ_EINVAL;
    if (d->rope_dims < 0 || d->rope_dims > d->head_dim) return FUSED_PROJ_EINVAL;
    Derived r;
    r.kvh = d->n_kv_heads > 0 ? d->n_kv_heads : d->n_heads;
    r.rd = d->rope_dims > 0 ? d->rope_dims : d->head_dim;
    if (r.rd % 2 != 0) return FUSED_PROJ_EINVAL;
    if (!(d->rope_base > 0.0) || !ok_number(d->rope_base) || !ok_number(d->magnitude)) return FUSED_PROJ_EINVAL;
    if (!(std::fabs(d->magnitude) < 3.0e38)) return FUSED_PROJ_EINVAL;   // fp32 in the kernel
    if (d->scaling != ROPE_SCALING_NONE && (!(d->factor > 0.0) || !ok_number(d->factor))) return FUSED_PROJ_EINVAL;
    if (d->scaling == ROPE_SCALING_BY_PARTS &&
        (!ok_number(d->low_turns) || !ok_number(d->high_turns) || !(d->low_turns < d->high_turns) ||
         d->original_tokens < 1))
        return FUSED_PROJ_EINVAL;
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (d->head_dim % 8 != 0 || d->head_dim > kMostDims) return FUSED_PROJ_EUNSUPPORTED;
    if (d->n_heads > (1 << 16) || d->n_heads + 2 * r.kvh > (1 << 16)) return FUSED_PROJ_EUNSUPPORTED;
    if (d->tokens > lim || d->batch > lim) return FUSED_PROJ_EUNSUPPORTED;
    if (d->batch * d->tokens > lim / d->head_dim) return FUSED_PROJ_EUNSUPPORTED;
    for (int64_t i = 0; i < r.rd / 2; ++i)
        if (!(pair_angle(*d, r.rd, i) <= kMostAngle)) return FUSED_PROJ_EUNSUPPORTED;
    r.rows = d->batch * d->tokens;
    const int v = d->dtype == FUSED_PROJ_BF16 ? 8 : 4;
    r.width = v;
    if (d->pairs == ROPE_PAIRS_HALF) {
        while ((r.rd / 2) % r.width != 0) r.width /= 2;
        r.units = (int)((d->head_dim - r.rd / 2) / r.width);
    } else {
        r.units = (int)(d->head_dim / v);
    }
    if (out) *out = r;
    return FUSED_PROJ_OK;
}

struct Range {
    uintptr_t lo, hi;
};
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }
Range range(const void* p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes}; }

int hip_status(hipError_t e) {
    if (e == hipSuccess) return FUSED_PROJ_OK;
    fp::set_last_hip_error(e);
    return FUSED_PROJ_EHIP;
}

}  // namespace

struct rope_plan {
    rope_desc d;
    Derived r;
    int device = -1;
    uint64_t* turns = nullptr;
};

namespace {

// Turns a position of every pair, as binary fractions without their whole turns.
void pair_turns(const rope_desc& d, int64_t rd, uint64_t (&f)[kMostDims / 2]) {
    for (int64_t i = 0; i < rd / 2; ++i) {
        const long double turns = pair_angle(d, rd, i) / kTwoPi;
        f[i] = (uint64_t)ldexpl(turns - floorl(turns), 64);
    }
}

// W: of a half's units; interleaved rows are taken in pieces of 16 bytes.
template <typename T, int W, int G>
void launch_heads(const RopeArgs& a, bool half, hipStream_t st) {
    const dim3 grid((unsigned)(((int64_t)a.items + 255) / 256), (unsigned)((a.heads + G - 1) / G));
    if (half)
        hipLaunchKernelGGL((rope_kernel<T, W, true, G>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((rope_kernel<T, (sizeof(T) == 2 ? 8 : 4), false, G>), grid, dim3(256), 0, st, a);
}
template <typename T, int W>
void launch(const RopeArgs& a, bool half, hipStream_t st) {
    if (((int64_t)a.items + 255) / 256 * ((a.heads + kHeads - 1) / kHeads) < kFewBlocks)
        launch_heads<T, W, 1>(a, half, st);
    else
        launch_heads<T, W, kHeads>(a, half, st);
}

int run(rope_t h, const Side& from, const Side& to, const int32_t* positions, bool with_v, bool backward, void* stream) {
    const rope_desc& d = h->d;
    const int esize = d.dtype == FUSED_PROJ_BF16 ? 2 : 4;
    const int parts = with_v ? 3 : 2;
    const int64_t head_bytes = h->r.rows * d.head_dim * esize;
    const int64_t heads[3] = {d.n_heads, h->r.kvh, h->r.kvh};
    Range in[4], out[3];
    int n_in = 0, n_out = 0;
    for (const Side* s : {&from, &to}) {
        for (int i = 0; i < (s->token_major ? 1 : parts); ++i) {
            if (!s->part[i]) return FUSED_PROJ_EINVAL;
            if ((uintptr_t)s->part[i] & 15u) return FUSED_PROJ_EALIGN;
            const Range r = range(s->part[i], (s->token_major ? d.n_heads + 2 * h->r.kvh : heads[i]) * head_bytes);
            (s == &from ? in[n_in++] : out[n_out++]) = r;
        }
    }
    if ((uintptr_t)positions & 3u) return FUSED_PROJ_EALIGN;
    const int tensors_in = n_in;
    if (positions) in[n_in++] = range(positions, h->r.rows * 4);
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (overlap(out[i], out[j])) return FUSED_PROJ_EALIAS;
        for (int j = 0; j < n_in; ++j) {
            // a rotation in place: the same tensor on both sides
            const bool same = !with_v && j < tensors_in && i == j && out[i].lo == in[j].lo;
            if (!same && overlap(out[i], in[j])) return FUSED_PROJ_EALIAS;
        }
    }
    int dev = -1;
    const int rc = hip_status(hipGetDevice(&dev));
    if (rc) return rc;
    if (dev != h->device) return FUSED_PROJ_EINVAL;
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.from = from;
    a.to = to;
    a.positions = positions;
    a.turns = h->turns;
    a.T = (int32_t)d.tokens;
    a.H = (int32_t)d.n_heads;
    a.KVH = (int32_t)h->r.kvh;
    a.hd = (int32_t)d.head_dim;
    a.rd = (int32_t)h->r.rd;
    a.heads = a.H + (with_v ? 2 : 1) * a.KVH;
    a.width = (int64_t)(d.n_heads + 2 * h->r.kvh) * d.head_dim;
    a.units = h->r.units;
    a.items = (uint32_t)(h->r.rows * h->r.units);
    a.grouped = d.qkv_order == FUSED_PROJ_QKV_GROUPED;
    a.backward = backward;
    a.magnitude = d.magnitude == 0.0 ? 1.0f : (float)d.magnitude;
    a.div_units = fp::make_fastdiv_u31((uint32_t)a.units);
    a.div_t = fp::make_fastdiv_u31((uint32_t)a.T);
    const bool half = d.pairs == ROPE_PAIRS_HALF;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (d.dtype == FUSED_PROJ_BF16) {
        switch (h->r.width) {
            case 8: launch<__bf16, 8>(a, half, st); break;
            case 4: launch<__bf16, 4>(a, half, st); break;
            case 2: launch<__bf16, 2>(a, half, st); break;
            default: launch<__bf16, 1>(a, half, st);
        }
    } else {
        switch (h->r.width) {
            case 4: launch<float, 4>(a, half, st); break;
            case 2: launch<float, 2>(a, half, st); break;
            default: launch<float, 1>(a, half, st);
        }
    }
    return hip_status(hipGetLastError());
}

Side heads_side(const void* q, const void* k, const void* v) {
    Side s;
    s.part[0] = (char*)q;
    s.part[1] = (char*)k;
    s.part[2] = (char*)v;
    s.token_major = 0;
    return s;
}
Side rows_side(const void* qkv) {
    Side s = heads_side(qkv, nullptr, nullptr);
    s.token_major = 1;
    return s;
}

}  // namespace

extern "C" {

int rope_validate(const rope_desc* desc) { return check(desc, nullptr); }

int rope_create(const rope_desc* desc, rope_t* out) {
    if (!out) return FUSED_PROJ_EINVAL;
    *out = nullptr;
    Derived r;
    int rc = check(desc, &r);
    if (rc) return rc;
    rope_plan* h = new (std::nothrow) rope_plan();
    if (!h) return FUSED_PROJ_EHIP;
    h->d = *desc;
    h->r = r;
    rc = hip_status(hipGetDevice(&h->device));
    if (!rc) {
        uint64_t f[kMostDims / 2];
        pair_turns(*desc, r.rd, f);
        const size_t bytes = (size_t)(r.rd / 2) * sizeof(uint64_t);
        rc = hip_status(hipMalloc((void**)&h->turns, bytes));
        if (!rc) rc = hip_status(hipMemcpy(h->turns, f, bytes, hipMemcpyHostToDevice));
    }
    if (rc) {
        rope_destroy(h);
        return rc;
    }
    *out = h;
    return FUSED_PROJ_OK;
}

int rope_split(rope_t h, const void* qkv, const int32_t* positions, void* q, void* k, void* v, void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (h->r.rows == 0) return FUSED_PROJ_OK;
    return run(h, rows_side(qkv), heads_side(q, k, v), positions, true, false, stream);
}

int rope_split_backward(rope_t h, const void* dq, const void* dk, const void* dv, const int32_t* positions, void* dqkv,
                        void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (h->r.rows == 0) return FUSED_PROJ_OK;
    return run(h, heads_side(dq, dk, dv), rows_side(dqkv), positions, true, true, stream);
}

int rope_rotate(rope_t h, const void* q, const void* k, const int32_t* positions, void* q_out, void* k_out,
                void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (h->r.rows == 0) return FUSED_PROJ_OK;
    return run(h, heads_side(q, k, nullptr), heads_side(q_out, k_out, nullptr), positions, false, false, stream);
}

int rope_rotate_backward(rope_t h, const void* dq_out, const void* dk_out, const int32_t* positions, void* dq, void* dk,
                         void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (h->r.rows == 0) return FUSED_PROJ_OK;
    return run(h, heads_side(dq_out, dk_out, nullptr), heads_side(dq, dk, nullptr), positions, false, true, stream);
}

int rope_destroy(rope_t h) {
    if (!h) return FUSED_PROJ_OK;
    const int rc = h->turns ? hip_status(hipFree(h->turns)) : FUSED_PROJ_OK;
    delete h;
    return rc;
}

}  // extern "C"
