// Attention over the key/value cache in 4 or 8 bits (gfx950; formulas and format are in
// include/kv_cache.h), on the bf16 matrix cores without dequantising.
//
// Codes as bf16 numbers. The bf16 number with the bits of a code c (0..255) is c 2^-133: the
// 7 mantissa bits of a denormal and the lowest exponent bit go on linearly, and the matrix
// cores take denormal inputs as they are. So a code becomes an operand by masking alone,
// and its products with q are exact. With 4 bits, every other code is masked where it lies,
// 4 bits up, and stands for 16 c 2^-133: those elements of q are divided by 16, those of the
// output at the end. q is multiplied by the power of two that brings the wave's largest value
// to 2^126, so that the products are ordinary numbers (sums of 256 stay below 2^11) and the
// factor that takes them back is small: it is multiplied by k's scales.
//
// The affine format stays outside the products. With a token's scale s and zero z,
//   q . khat = s (q . c) + z sum(q)
//   sum_j p_j vhat_j = sum_j b_j (c_j - C) + sum_j p_j (z_j + C s_j),    b_j = p_j s_j in bf16
// The second sum is kept apart from the codes' powers of two: zero has no bound as s has one.
// C is the middle code: codes are positive, so the rounding of b_j times c_j would be that of
// a sum far larger than the result; times c_j - C it is the rounding of the values' own
// spread (measured: output error 0.0023 of the output's norm instead of 0.0049, of which
// 0.0017 is the output's own rounding). C sum_j b_j is one more product, with a constant.
//
// Tiles. A wave holds R x 16 query rows (all rows of a k/v head: token by token, its group's
// heads inside) and takes 32 positions at a time, two halves of 16 that each lie in one
// page. S = K Q^T (16 positions x 16 rows a product) leaves each lane 4 positions of one
// row, which is the operand layout of O^T = V^T P^T if the 32 positions of that product are
// counted as the lanes hold them: nothing is exchanged between lanes but row maxima. K's
// operand is contiguous in memory up to a permutation of the head's elements, which q's
// operand shares. V's operand needs 8 positions of one element in a lane: a lane reads the
// same few bytes of 8 positions and pairs them up with byte permutes.
//
// Measured, 4 bits, 32 heads on 8 x 128: 63 sequences of 8191 positions, one token each, 106 us
// (5.2 TB/s, a large copy's rate); of 2500 to 8191 positions 80 us (48% of the vector pipes'
// time); 2 x 1024 tokens over 4096 positions 180 us (670 TFLOP/s; a large bf16 product reaches
// 1209).
#include <cmath>

#include "kv_cache.h"
#include "vector_io.h"

namespace {

using namespace fp::dev;
using fp::CacheArgs;

constexpr float kLowest = -3.0e38f;   // the running maximum before any position
// Probabilities are held times 2^-24: zero + C scale may be any bfloat16 number (a row of one value
// is kept whatever its size), and the largest, under probabilities of up to 2^kSlack, still adds up
// over 2^16 positions, while numbers down to 2^-117 keep the 8 bits that o has. v's scales (at most
// 2^24) are taken times 2^103 instead: their products with probabilities and codes of 2^-133
// neither overflow nor vanish.
constexpr float kLift = -24.0f;
constexpr uint32_t kScaleLift = 103;
constexpr float kSlack = 8.0f;        // how far (log2) a logit may pass the running maximum before it moves

template <int D, int BITS>
struct Shape {
    static constexpr int ROWB = D * BITS / 8;            // bytes of a row
    static constexpr int KS = D / 32;                    // products over a head's elements
    static constexpr int KW = ROWB / 16;                 // words of K a lane reads (a quarter row)
    // V: the head in parts of a power of two; of each part a lane reads B bytes a position
    static constexpr int D0 = D >= 256 ? 256 : D >= 128 ? 128 : D >= 64 ? 64 : 32, D1 = D - D0;
    static constexpr int B0 = D0 / 16 * BITS / 8, B1 = D1 / 16 * BITS / 8;
    static constexpr int W0 = (B0 + 3) / 4, W1 = (B1 + 3) / 4;
    static constexpr int NT = D / 16;                    // output tiles
};

// What a lane reads of 32 positions.
template <int D, int BITS>
struct Tile {
    using Sh = Shape<D, BITS>;
    uint32_t k[2][Sh::KW];                       // position 16 u + lane % 16, quarter lane / 16 of the row
    uint32_t v0[2][4][Sh::W0];                   // position 16 u + 4 (lane / 16) + j
    uint32_t v1[2][4][Sh::W1 > 0 ? Sh::W1 : 1];
    u32x4 kp[2], vp[2];                          // their params
    int32_t known[2];                            // positions of the half that exist (0..16)
};

// B bytes (1, 2 or whole words) into words.
template <int B>
__device__ __forceinline__ void load_bytes(uint32_t* w, const uint8_t* p) {
    if constexpr (B == 1)
        w[0] = *p;
    else if constexpr (B == 2)
        w[0] = *reinterpret_cast<const uint16_t*>(p);
    else
        __builtin_memcpy(w, __builtin_assume_aligned(p, 4), B);
}

// The pages of a tile's halves, by scalar loads: a tile's own loads wait for them alone.
struct Pages {
    int32_t id[2];
};
__device__ __forceinline__ Pages pages_of(const CacheArgs& a, const int32_t* table, int tile, int length) {
    typedef const __attribute__((address_space(4))) int32_t* scalar;
    Pages g;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int p = tile * 32 + u * 16;
        g.id[u] = ((scalar)table)[fp::fastdiv_u31((uint32_t)(p < length ? p : 0), a.div_page)];
    }
    return g;
}

template <int D, int BITS>
__device__ __forceinline__ void load_tile(Tile<D, BITS>& t, const CacheArgs& a, const Pages& g, int kvh, int tile, int length) {
    using Sh = Shape<D, BITS>;
    const int lane = threadIdx.x & 63, m = lane & 15, qd = lane >> 4;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int p = tile * 32 + u * 16;
        const bool there = p < length && (uint32_t)g.id[u] < (uint32_t)a.n_pages;
        const int in_page = p - (int)fp::fastdiv_u31((uint32_t)p, a.div_page) * a.page_size;
        // any row that exists stands in for one that does not
        const int64_t row = there ? (int64_t)g.id[u] * a.page_rows + ((int64_t)kvh * a.page_size + in_page) : 0;
        t.known[u] = there ? (length - p < 16 ? length - p : 16) : 0;
        const uint8_t* kc = a.k_codes + row * Sh::ROWB;
        const uint8_t* vc = a.v_codes + row * Sh::ROWB;
        load_bytes<Sh::KW * 4>(t.k[u], kc + (uint32_t)(m * Sh::ROWB + qd * (Sh::ROWB / 4)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            load_bytes<Sh::B0>(t.v0[u][j], vc + (uint32_t)((qd * 4 + j) * Sh::ROWB + m * Sh::B0));
            if constexpr (Sh::D1 > 0)
                load_bytes<Sh::B1>(t.v1[u][j], vc + (uint32_t)((qd * 4 + j) * Sh::ROWB + Sh::D0 * BITS / 8 + m * Sh::B1));
        }
        t.kp[u] = *reinterpret_cast<const u32x4*>(a.k_params + row + (uint32_t)(qd * 4));
        t.vp[u] = *reinterpret_cast<const u32x4*>(a.v_params + row + (uint32_t)(qd * 4));
    }
}

__device__ __forceinline__ float param_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float param_zero(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 8 codes as an operand. Order of the elements: 0 4 1 5 2 6 3 7 (4 bits; 1 5 3 7 times 16)
// or 0 2 1 3 4 6 5 7 (8 bits).
template <int BITS>
__device__ __forceinline__ bf16x8 codes_operand(const uint32_t* w) {
    u32x4 r;
    if constexpr (BITS == 4) {
        const uint32_t lo = w[0], hi = w[0] >> 8;
        r = u32x4{lo & 0x000F000Fu, lo & 0x00F000F0u, hi & 0x000F000Fu, hi & 0x00F000F0u};
    } else {
        r = u32x4{w[0] & 0x00FF00FFu, (w[0] >> 8) & 0x00FF00FFu, w[1] & 0x00FF00FFu, (w[1] >> 8) & 0x00FF00FFu};
    }
    return __builtin_bit_cast(bf16x8, r);
}
template <int BITS>
__device__ constexpr int operand_element(int i) {
    return BITS == 4 ? (i >> 1) + 4 * (i & 1) : (i & 4) + ((i >> 1) & 1) + 2 * (i & 1);
}

__device__ __forceinline__ float max_over_quads(float v) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_over_quads(float v) { return swap_sum32(swap_sum16(v, v), swap_sum16(v, v)); }

// A wave's running state.
template <int D, int R>
struct State {
    f32x4 o[R][D / 16];    // output tiles, in codes: see each_run
    f32x4 c[R];               // 2 C sum_j b_j, in codes: the same in all four
    float m[R], l[R], z[R];   // running maximum (log2), and this lane's sums of p and of p (z + C s), times 2^-24
};
template <int D, int R>
__device__ __forceinline__ void clear(State<D, R>& st) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        st.m[r] = kLowest;
        st.l[r] = st.z[r] = 0.0f;
        st.c[r] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[r][i] = f32x4{0, 0, 0, 0};
    }
}

// The affine part of a lane's 8 positions (two halves of 4): k's scale times the logits'
// factor, k's zero, v's scale times 2^103, v's zero + C times its scale.
struct Affine {
    float ks[2][4], kz[2][4], vs[2][4], vz[2][4];
};
// By the exponent, with the shift that unpacks it: a scale of 0 or a denormal one becomes another of
// 2^-126 or less, here and in `middle`. A NaN becomes a number: its row's zero is NaN too.
__device__ __forceinline__ float lifted_scale(uint32_t w) { return __uint_as_float((w << 16) + (kScaleLift << 23)); }
template <int BITS>
__device__ __forceinline__ float middle(uint32_t w) {
    static_assert(kScaleLift == 103, "the factor that takes the lift back");
    return fmaf(lifted_scale(w), 0x1p-103f * 0.5f * (float)((1 << BITS) - 1), param_zero(w));
}

// What hides positions from the wave's rows: the halves' existing positions, the tile's first
// position and each row's own.
template <int R>
struct Sight {
    int known[2], at;
    int last[R], first_last;
};

// Probabilities (bf16, times v's scale) of 32 positions from the products s of codes and
// queries; moves the running maximum where a logit passes it by more than kSlack. Masks cost
// more than the rest together, so a tile takes them only where some row of the wave does not
// see some position, in branches of their own (kept from being turned into selects).
template <int D, int R>
__device__ __forceinline__ void probabilities(State<D, R>& st, bf16x8 (&p)[R], const f32x4 (&s)[R][2], const Affine& af,
                                              const float (&zq)[R], const Sight<R>& sg) {
    const int qd = (threadIdx.x & 63) >> 4;
    const bool edge = sg.known[0] < 16 || sg.known[1] < 16 || sg.at + 31 > sg.first_last;
    const auto seen = [&](int r, int u, int i) {
        return qd * 4 + i < sg.known[u] && sg.at + u * 16 + qd * 4 + i <= sg.last[r];
    };
    float y[R][2][4];
    const auto each = [&](auto f) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) f(r, u, i);
    };
    const auto hide = [&]() {
        if (edge) {
            asm volatile("");
            each([&](int r, int u, int i) { y[r][u][i] = seen(r, u, i) ? y[r][u][i] : -INFINITY; });
        }
    };
    const auto greatest = [&](int r) {
        float top = fmaxf(y[r][0][0], y[r][0][1]);
#pragma unroll
        for (int k = 2; k < 8; ++k) top = fmaxf(top, y[r][k >> 2][k & 3]);
        return top;
    };
    float base[R];
#pragma unroll
    for (int r = 0; r < R; ++r) base[r] = kLift - st.m[r];
    each([&](int r, int u, int i) { y[r][u][i] = fmaf(af.ks[u][i], s[r][u][i], fmaf(af.kz[u][i], zq[r], base[r])); });
    hide();
    float top = greatest(0);
#pragma unroll
    for (int r = 1; r < R; ++r) top = fmaxf(top, greatest(r));
    if (__any(top > kLift + kSlack)) {
        // the maximum moves: the logits again, without the old one
        each([&](int r, int u, int i) { y[r][u][i] = fmaf(af.ks[u][i], s[r][u][i], af.kz[u][i] * zq[r]); });
        hide();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float m = fmaxf(st.m[r], max_over_quads(greatest(r)));
            const float down = __builtin_amdgcn_exp2f(st.m[r] - m);
            st.m[r] = m;
            st.l[r] *= down;
            st.z[r] *= down;
            st.c[r] *= down;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) st.o[r][i] *= down;
        }
        each([&](int r, int u, int i) { y[r][u][i] = (y[r][u][i] - st.m[r]) + kLift; });
    }
    each([&](int r, int u, int i) {
        y[r][u][i] = __builtin_amdgcn_exp2f(y[r][u][i]);
        st.l[r] += y[r][u][i];
    });
    if (edge) {
        asm volatile("");
        each([&](int r, int u, int i) {
            // what a row does not see may be NaN
            const bool sees = seen(r, u, i);
            p[r][u * 4 + i] = (__bf16)(sees ? y[r][u][i] * af.vs[u][i] : 0.0f);
            st.z[r] = fmaf(y[r][u][i], sees ? af.vz[u][i] : 0.0f, st.z[r]);
        });
    } else {
        asm volatile("");
        each([&](int r, int u, int i) {
            p[r][u * 4 + i] = (__bf16)(y[r][u][i] * af.vs[u][i]);
            st.z[r] = fmaf(y[r][u][i], af.vz[u][i], st.z[r]);
        });
    }
}

template <int D, int BITS, int R>
__device__ __forceinline__ void count_middle(State<D, R>& st, const bf16x8 (&p)[R]) {
    constexpr uint32_t kTwiceC = ((1u << BITS) - 1) * 0x00010001u;
    const bf16x8 twice_c = __builtin_bit_cast(bf16x8, u32x4{kTwiceC, kTwiceC, kTwiceC, kTwiceC});
#pragma unroll
    for (int r = 0; r < R; ++r) st.c[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(twice_c, p[r], st.c[r], 0, 0, 0);
}

// Pairs of positions: byte b of two words, each in the low half of 16 bits.
__device__ __forceinline__ uint32_t byte_pair(uint32_t first, uint32_t second, int b) {
    return __builtin_amdgcn_perm(second, first, 0x0C040C00u + 0x00010001u * b);
}

template <int D, int BITS, int R>
__device__ __forceinline__ void take_tile(State<D, R>& st, const Tile<D, BITS>& t, const bf16x8 (&q)[R][D / 32],
                                          const float (&zq)[R], const int (&last)[R], int first_last, float c1, int tile) {
    using Sh = Shape<D, BITS>;
    Affine af;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            af.ks[u][i] = param_scale(t.kp[u][i]) * c1;
            af.kz[u][i] = param_zero(t.kp[u][i]);
            af.vs[u][i] = lifted_scale(t.vp[u][i]);
            af.vz[u][i] = middle<BITS>(t.vp[u][i]);
        }
    f32x4 s[R][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][u] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < Sh::KS; ++j) {
            const bf16x8 k = codes_operand<BITS>(&t.k[u][j * BITS / 4]);
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[r][j], s[r][u], 0, 0, 0);
        }
    }
    Sight<R> sg;
    sg.known[0] = t.known[0];
    sg.known[1] = t.known[1];
    sg.at = tile * 32;
    sg.first_last = first_last;
#pragma unroll
    for (int r = 0; r < R; ++r) sg.last[r] = last[r];
    bf16x8 p[R];
    probabilities<D, R>(st, p, s, af, zq, sg);
    count_middle<D, BITS, R>(st, p);
    const auto part = [&](auto bytes, auto first, const auto& w) {
        constexpr int B = decltype(bytes)::value, T0 = decltype(first)::value;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            u32x4 x;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) x[u * 2 + h] = byte_pair(w[u][2 * h][b >> 2], w[u][2 * h + 1][b >> 2], b & 3);
            if constexpr (BITS == 8) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    st.o[r][T0 + b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), p[r], st.o[r][T0 + b], 0, 0, 0);
            } else {
                const bf16x8 lo = __builtin_bit_cast(bf16x8, x & 0x000F000Fu), hi = __builtin_bit_cast(bf16x8, x & 0x00F000F0u);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    st.o[r][T0 + 2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, p[r], st.o[r][T0 + 2 * b], 0, 0, 0);
                    st.o[r][T0 + 2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, p[r], st.o[r][T0 + 2 * b + 1], 0, 0, 0);
                }
            }
        }
    };
    part(std::integral_constant<int, Sh::B0>{}, std::integral_constant<int, 0>{}, t.v0);
    if constexpr (Sh::D1 > 0) part(std::integral_constant<int, Sh::B1>{}, std::integral_constant<int, Sh::D0 / 16>{}, t.v1);
}

// Calls f(d, values) for each run of consecutive elements d .. d + N - 1 that the lane holds of
// its row, still to be divided by the row's sum (both times 2^-24). The lift ends here: codes of
// 2^-133 times scales of 2^103 come back by 2^30 (the 4-bit codes masked 4 bits up by 2^26).
template <int D, int BITS, int R, typename F>
__device__ __forceinline__ void each_run(const State<D, R>& st, int r, float z, F f) {
    using Sh = Shape<D, BITS>;
    const int qd = (threadIdx.x & 63) >> 4;
    const auto part = [&](auto size, auto first) {
        constexpr int N = decltype(size)::value / 16, T0 = decltype(first)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[N];
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = fmaf(st.o[r][T0 + k][i], BITS == 4 && (k & 1) ? 0x1p26f : 0x1p30f, z);
            f(T0 * 16 + (qd * 4 + i) * N, v);
        }
    };
    part(std::integral_constant<int, Sh::D0>{}, std::integral_constant<int, 0>{});
    if constexpr (Sh::D1 > 0) part(std::integral_constant<int, Sh::D1>{}, std::integral_constant<int, Sh::D0 / 16>{});
}

// N (2 or a multiple of 4) values to bf16 at p.
template <int N>
__device__ __forceinline__ void store_bf16(__bf16* p, const float* v) {
    typedef __bf16 bf16xn __attribute__((ext_vector_type(N)));
    bf16xn o;
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = (__bf16)v[k];
    *reinterpret_cast<bf16xn*>(p) = o;
}

// A wave's query rows: R x 16 of the rows of a k/v head, from row0 on.
template <int D, int BITS, int R>
struct Rows {
    int last[R];              // this lane's row: the last position it sees (-1: none)
    int out[R];               // its place in o, b T H of them (31 bits)
    bool real[R];
    int first_last;           // the last position that all rows see (below 0: some see none)
    int sees;                 // positions that any row sees
    bf16x8 q[R][D / 32];      // the operand: q times 2^lift
    float zq[R];              // sum q times the logits' factor
};

// The rows' places and their own positions, and their queries' bits; returns the largest
// exponent field among the lane's rows whose values are all below q_limit (others give NaN).
template <int D, int BITS, int R>
__device__ __forceinline__ uint32_t find_rows(Rows<D, BITS, R>& w, u32x4 (&raw)[R][D / 32], bool (&bad)[R], const CacheArgs& a,
                                              const fp::Step& step, int seq, int kvh, int row0) {
    const int lane = threadIdx.x & 63, n = lane & 15, qd = lane >> 4, rows = a.group * a.T;
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * 16 + n;
        w.real[r] = row < rows;
        const int s = w.real[r] ? (int)fp::fastdiv_u31((uint32_t)row, a.div_group) : 0, h = w.real[r] ? row - s * a.group : 0;
        w.last[r] = w.real[r] && s < step.count ? step.first + s : -1;
        const int qh = kvh * a.group + h;
        w.out[r] = (seq * a.T + s) * a.H + qh;
        const __bf16* q = static_cast<const __bf16*>(a.q) + ((int64_t)(seq * a.H + qh) * a.T + s) * D + qd * (D / 4);
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            raw[r][j] = w.real[r] ? *reinterpret_cast<const u32x4*>(q + j * 8) : u32x4{0, 0, 0, 0};
            // padding sees nothing: what lies there takes no part, in the lift neither (behind the load,
            // which does not wait for the sequence's lengths)
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[r][j][i] = w.last[r] >= 0 ? raw[r][j][i] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) mine = max(mine, max((raw[r][j][i] >> 7) & 0xFFu, (raw[r][j][i] >> 23) & 0xFFu));
        }
        mine = max(mine, (uint32_t)__shfl_xor((int)mine, 16));
        mine = max(mine, (uint32_t)__shfl_xor((int)mine, 32));
        bad[r] = mine >= (uint32_t)a.q_limit;
        top = max(top, bad[r] ? 0u : mine);
    }
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, k));
    // rows are token by token: the wave's first and last token of the step
    const int s_first = (int)fp::fastdiv_u31((uint32_t)(row0 < rows ? row0 : 0), a.div_group);
    const int row_end = min(row0 + R * 16, rows) - 1;
    const int s_last = min((int)fp::fastdiv_u31((uint32_t)max(row_end, 0), a.div_group), step.count - 1);
    const bool any = row0 < rows && s_first < step.count;
    w.first_last = any && s_last * a.group + a.group - 1 >= row_end ? step.first + s_first : -1;
    w.sees = any ? max(min(step.length, step.first + s_last + 1), 0) : 0;
    return top;
}
template <int D, int BITS, int R>
__device__ __forceinline__ void lift_rows(Rows<D, BITS, R>& w, const u32x4 (&raw)[R][D / 32], const bool (&bad)[R], int lift,
                                          float logit_scale) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = bad[r] ? 0.0f : Piece<__bf16>::get(raw[r][j], operand_element<BITS>(i));
                sum += f;
                w.q[r][j][i] = (__bf16)ldexpf(f, BITS == 4 && (i & 2) ? lift - 4 : lift);   // exact
            }
        }
        sum = sum_over_quads(sum);
        w.zq[r] = bad[r] ? NAN : sum * logit_scale;
    }
}
// q's lift that brings the exponent field `top` to 2^126, and the factor that takes the products
// back: 2^(7 + e) logit_scale for a largest value of 2^e, at most 2^103 by q_limit. With k's scale
// (at most 2^24) that is a finite number for every row, whatever row of the workgroup is largest.
__device__ __forceinline__ int lift_of(uint32_t top) { return 126 - ((int)max(top, 1u) - 127); }
__device__ __forceinline__ float logits_factor(int lift, float logit_scale) { return ldexpf(logit_scale, 133 - lift); }

// Which part of the work a workgroup takes. k/v heads run fastest: the workgroups of one
// share an XCD's L2 where their number is a multiple of 8; the last rows, which see the
// most, come first. The second half of the grid takes the sequences backwards: a CU that
// holds a workgroup of each half rarely has two of the longest sequence.
struct Share {
    int seq, kvh, block, split;
};
__device__ __forceinline__ Share share_of(const CacheArgs& a) {
    const int heads = a.batch * a.KVH;
    const int head = (int)(blockIdx.x % (uint32_t)heads), rest = (int)(blockIdx.x / (uint32_t)heads);
    Share s;
    s.split = (int)fp::fastdiv_u31((uint32_t)rest, a.div_blocks);
    s.block = a.row_blocks - 1 - (rest - s.split * a.row_blocks);
    s.seq = (int)fp::fastdiv_u31((uint32_t)head, a.div_kvh);
    s.kvh = head - s.seq * a.KVH;
    if (2 * rest >= a.row_blocks * a.splits) s.seq = a.batch - 1 - s.seq;
    return s;
}

// Few rows (single and drafted tokens): the four waves of a workgroup hold the same R x 16
// rows and take different positions, each by itself; at the end they are put together in
// LDS. Bound by the cache's bytes: the next tile is loaded while one is taken.
//
// Waves a SIMD: as many as the registers of two tiles and the output leave; 8 bits with heads of
// 128 and two row tiles spill 20 bytes a lane at two waves, 8 bits with heads of 256 take
// accumulation registers besides, and one wave.
template <int D, int BITS, int R>
constexpr int kStepWaves = D * BITS > 1536 ? 1 : D * BITS <= 512 && R == 1 && Shape<D, BITS>::D1 == 0 ? 3 : 2;

template <int D, int BITS, int R>
__global__ __launch_bounds__(256, (kStepWaves<D, BITS, R>)) void kv_attend_kernel(CacheArgs a) {
    constexpr int WT = 4, PAD = D + 4;
    __shared__ float both[WT * 16 * PAD];
    __shared__ float both_ml[WT * 16 * 2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, n = lane & 15, qd = lane >> 4;
    const Share sh = share_of(a);
    const fp::Step step = fp::step_of(a, sh.seq);
    const int rows = a.group * a.T, row0 = sh.block * R * 16;
    Rows<D, BITS, R> w;
    float c1;
    {
        u32x4 raw[R][D / 32];
        bool bad[R];
        const int lift = lift_of(find_rows<D, BITS, R>(w, raw, bad, a, step, sh.seq, sh.kvh, row0));
        lift_rows<D, BITS, R>(w, raw, bad, lift, a.logit_scale);
        c1 = logits_factor(lift, a.logit_scale);
    }
    const int tiles = (w.sees + 31) >> 5, per = (tiles + a.splits - 1) / a.splits;
    const int t_begin = sh.split * per, t_end = min(tiles, t_begin + per);

    State<D, R> st;
    clear<D, R>(st);
    const int32_t* table = a.table + (int64_t)sh.seq * a.max_pages;
    // two tiles in turn: one is loaded while the other is taken, and the pages of the next are
    // known before that. Tiles past the end load a row that exists and are not taken.
    int tile = t_begin + wave;
    if (tile < t_end) {
        Tile<D, BITS> even, odd;
        load_tile<D, BITS>(even, a, pages_of(a, table, tile, step.length), sh.kvh, tile, step.length);
        Pages next = pages_of(a, table, tile + WT, step.length);
        while (true) {
            load_tile<D, BITS>(odd, a, next, sh.kvh, tile + WT, step.length);
            next = pages_of(a, table, tile + 2 * WT, step.length);
            take_tile<D, BITS, R>(st, even, w.q, w.zq, w.last, w.first_last, c1, tile);
            tile += WT;
            if (tile >= t_end) break;
            load_tile<D, BITS>(even, a, next, sh.kvh, tile + WT, step.length);
            next = pages_of(a, table, tile + 2 * WT, step.length);
            take_tile<D, BITS, R>(st, odd, w.q, w.zq, w.last, w.first_last, c1, tile);
            tile += WT;
            if (tile >= t_end) break;
        }
    }

#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float l = sum_over_quads(st.l[r]);
        const float z = fmaf(st.c[r][0], -0x1p29f, sum_over_quads(st.z[r]));
        // the workgroup's waves together, 16 rows at a time
        if (r > 0) __syncthreads();
        float* mine = both + (wave * 16 + n) * PAD;
        each_run<D, BITS, R>(st, r, z, [&](int d, auto& v) {
            constexpr int N = sizeof(v) / 4;
#pragma unroll
            for (int k = 0; k < N; ++k) mine[d + k] = v[k];
        });
        if (qd == 0) {
            both_ml[(wave * 16 + n) * 2] = st.m[r];
            both_ml[(wave * 16 + n) * 2 + 1] = l;
        }
        __syncthreads();
        for (int it = threadIdx.x; it < 16 * (D / 8); it += 256) {
            const int rr = it / (D / 8), d = it % (D / 8) * 8, row = row0 + r * 16 + rr;
            if (row >= rows) continue;
            const int s = (int)fp::fastdiv_u31((uint32_t)row, a.div_group), qh = sh.kvh * a.group + row - s * a.group;
            const int64_t out = (int64_t)(sh.seq * a.T + s) * a.H + qh;
            float m = kLowest, f[WT], sum = 0.0f, v[8];
#pragma unroll
            for (int k = 0; k < WT; ++k) m = fmaxf(m, both_ml[(k * 16 + rr) * 2]);
#pragma unroll
            for (int k = 0; k < WT; ++k) {
                f[k] = __builtin_amdgcn_exp2f(both_ml[(k * 16 + rr) * 2] - m);
                sum = fmaf(f[k], both_ml[(k * 16 + rr) * 2 + 1], sum);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = 0.0f;
#pragma unroll
                for (int k = 0; k < WT; ++k) v[e] = fmaf(f[k], both[(k * 16 + rr) * PAD + d + e], v[e]);
            }
            if (a.splits == 1) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= inv;
                store_bf16<8>(static_cast<__bf16*>(a.o) + out * D + d, v);
            } else {
                const int64_t at = (int64_t)sh.split * a.batch * a.T * a.H + out;
                if (d == 0) {
                    a.part_ml[at * 2] = m;
                    a.part_ml[at * 2 + 1] = sum;
                }
                if (t_begin >= t_end) continue;   // an empty part: its sum is 0, its values are not read
                f32x4* po = reinterpret_cast<f32x4*>(a.part_o + at * D + d);
                po[0] = f32x4{v[0], v[1], v[2], v[3]};
                po[1] = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
    }
}

// Many rows (a prompt's chunk): the NW waves of a workgroup hold different rows and take the
// same positions, 16 NW at a time. Bound by the softmax's vector work, so the operands are
// made once for all waves: each makes those of its 16 positions and puts them in LDS (the
// matrix cores' operand layout, 16 bytes a lane), two sets in turn with one barrier each,
// and the bytes of the positions after next are already under way.
template <int D, int BITS, int NW>
struct Shared {
    using Sh = Shape<D, BITS>;
    u32x4 k[NW][Sh::KS][64];        // a half's K operands
    u32x4 v[NW / 2][Sh::NT][64];    // 32 positions' V operands
    float affine[4][NW * 16];
    int known[NW];
};

template <int D, int BITS>
struct Raw {
    using Sh = Shape<D, BITS>;
    uint32_t k[Sh::KW], v0[4][Sh::W0], v1[4][Sh::W1 > 0 ? Sh::W1 : 1], kp, vp;
    int known;
};

template <int D, int BITS>
__device__ __forceinline__ void load_raw(Raw<D, BITS>& t, const CacheArgs& a, int page, int kvh, int p, int length) {
    using Sh = Shape<D, BITS>;
    const int lane = threadIdx.x & 63, m = lane & 15, qd = lane >> 4;
    const bool there = p < length && (uint32_t)page < (uint32_t)a.n_pages;
    const int in_page = p - (int)fp::fastdiv_u31((uint32_t)p, a.div_page) * a.page_size;
    const int64_t row = there ? (int64_t)page * a.page_rows + ((int64_t)kvh * a.page_size + in_page) : 0;
    t.known = there ? (length - p < 16 ? length - p : 16) : 0;
    const uint8_t* kc = a.k_codes + row * Sh::ROWB;
    const uint8_t* vc = a.v_codes + row * Sh::ROWB;
    load_bytes<Sh::KW * 4>(t.k, kc + (uint32_t)(m * Sh::ROWB + qd * (Sh::ROWB / 4)));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        load_bytes<Sh::B0>(t.v0[j], vc + (uint32_t)((qd * 4 + j) * Sh::ROWB + m * Sh::B0));
        if constexpr (Sh::D1 > 0)
            load_bytes<Sh::B1>(t.v1[j], vc + (uint32_t)((qd * 4 + j) * Sh::ROWB + Sh::D0 * BITS / 8 + m * Sh::B1));
    }
    t.kp = a.k_params[row + (uint32_t)m];
    t.vp = a.v_params[row + (uint32_t)m];
}

template <int D, int BITS, int NW>
__device__ __forceinline__ void share_raw(Shared<D, BITS, NW>& to, const Raw<D, BITS>& t, int wave, float c1) {
    using Sh = Shape<D, BITS>;
    const int lane = threadIdx.x & 63, u = wave & 1;
#pragma unroll
    for (int j = 0; j < Sh::KS; ++j) to.k[wave][j][lane] = __builtin_bit_cast(u32x4, codes_operand<BITS>(&t.k[j * BITS / 4]));
    const auto part = [&](auto bytes, auto first, const auto& w) {
        constexpr int B = decltype(bytes)::value, T0 = decltype(first)::value;
        const auto put = [&](int tile, u32x2 x) { reinterpret_cast<u32x2*>(&to.v[wave >> 1][tile][lane])[u] = x; };
#pragma unroll
        for (int b = 0; b < B; ++b) {
            u32x2 x;
#pragma unroll
            for (int h = 0; h < 2; ++h) x[h] = byte_pair(w[2 * h][b >> 2], w[2 * h + 1][b >> 2], b & 3);
            if constexpr (BITS == 8) {
                put(T0 + b, x);
            } else {
                put(T0 + 2 * b, x & 0x000F000Fu);
                put(T0 + 2 * b + 1, x & 0x00F000F0u);
            }
        }
    };
    part(std::integral_constant<int, Sh::B0>{}, std::integral_constant<int, 0>{}, t.v0);
    if constexpr (Sh::D1 > 0) part(std::integral_constant<int, Sh::B1>{}, std::integral_constant<int, Sh::D0 / 16>{}, t.v1);
    if (lane < 16) {
        to.affine[0][wave * 16 + lane] = param_scale(t.kp) * c1;
        to.affine[1][wave * 16 + lane] = param_zero(t.kp);
        to.affine[2][wave * 16 + lane] = lifted_scale(t.vp);
        to.affine[3][wave * 16 + lane] = middle<BITS>(t.vp);
    }
    if (lane == 0) to.known[wave] = t.known;
}

template <int D, int BITS, int R, int NW, int SETS>
__global__ __launch_bounds__(NW * 64, 2) void kv_attend_chunk_kernel(CacheArgs a) {
    using Sh = Shape<D, BITS>;
    constexpr int STEP = NW * 16;
    __shared__ Shared<D, BITS, NW> sets[SETS];
    __shared__ uint32_t tops[NW];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, qd = lane >> 4;
    const Share sh = share_of(a);
    const fp::Step step = fp::step_of(a, sh.seq);
    Rows<D, BITS, R> w;
    float c1;
    {
        u32x4 raw[R][D / 32];
        bool bad[R];
        const uint32_t mine = find_rows<D, BITS, R>(w, raw, bad, a, step, sh.seq, sh.kvh, (sh.block * NW + wave) * R * 16);
        if (lane == 0) tops[wave] = mine;
        __syncthreads();
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < NW; ++k) top = max(top, tops[k]);
        const int lift = lift_of(top);   // one for the workgroup: K's affine part is shared
        lift_rows<D, BITS, R>(w, raw, bad, lift, a.logit_scale);
        c1 = logits_factor(lift, a.logit_scale);
    }
    // the workgroup's positions: those of its last real row
    const int rows = a.group * a.T, row_end = min((sh.block + 1) * NW * R * 16, rows) - 1;
    const int s_last = min((int)fp::fastdiv_u31((uint32_t)row_end, a.div_group), step.count - 1);
    const int s_first = (int)fp::fastdiv_u31((uint32_t)(sh.block * NW * R * 16), a.div_group);
    const int sees = s_first < step.count ? max(min(step.length, step.first + s_last + 1), 0) : 0;
    const int turns = (sees + STEP - 1) / STEP, per = (turns + a.splits - 1) / a.splits;
    const int t_begin = sh.split * per, t_end = min(turns, t_begin + per);

    State<D, R> st;
    clear<D, R>(st);
    if (t_begin < t_end) {
        typedef const __attribute__((address_space(4))) int32_t* scalar;
        const scalar table = (scalar)(a.table + (int64_t)sh.seq * a.max_pages);
        const auto place = [&](int turn) { return turn * STEP + wave * 16; };
        const auto page_of = [&](int turn) {
            const int p = place(turn);
            return table[fp::fastdiv_u31((uint32_t)(p < step.length ? p : 0), a.div_page)];
        };
        Raw<D, BITS> raw;
        load_raw<D, BITS>(raw, a, page_of(t_begin), sh.kvh, place(t_begin), step.length);
        share_raw<D, BITS, NW>(sets[0], raw, wave, c1);
        load_raw<D, BITS>(raw, a, page_of(t_begin + 1), sh.kvh, place(t_begin + 1), step.length);
        int page = page_of(t_begin + 2);
        __syncthreads();
        for (int turn = t_begin; turn < t_end; ++turn) {
            const Shared<D, BITS, NW>& now = sets[(turn - t_begin) % SETS];
            const auto prepare_next = [&]() {
                if (turn + 1 < t_end) share_raw<D, BITS, NW>(sets[(turn + 1 - t_begin) % SETS], raw, wave, c1);
                load_raw<D, BITS>(raw, a, page, sh.kvh, place(turn + 2), step.length);
                page = page_of(turn + 3);
            };
            if constexpr (SETS == 2) prepare_next();   // the other set was read before the last barrier
#pragma unroll 1
            for (int g = 0; g < NW / 2; ++g) {
                Sight<R> sg;
                sg.at = turn * STEP + g * 32;
                if (sg.at >= w.sees) break;   // this wave's rows see nothing from here on
                sg.known[0] = __builtin_amdgcn_readfirstlane(now.known[2 * g]);
                sg.known[1] = __builtin_amdgcn_readfirstlane(now.known[2 * g + 1]);
                sg.first_last = w.first_last;
#pragma unroll
                for (int r = 0; r < R; ++r) sg.last[r] = w.last[r];
                f32x4 s[R][2];
                Affine af;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int r = 0; r < R; ++r) s[r][u] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < Sh::KS; ++j) {
                        const bf16x8 k = __builtin_bit_cast(bf16x8, now.k[2 * g + u][j][lane]);
#pragma unroll
                        for (int r = 0; r < R; ++r) s[r][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, w.q[r][j], s[r][u], 0, 0, 0);
                    }
                    const int at = (2 * g + u) * 16 + qd * 4;
                    const f32x4 ks = *reinterpret_cast<const f32x4*>(&now.affine[0][at]), kz = *reinterpret_cast<const f32x4*>(&now.affine[1][at]);
                    const f32x4 vs = *reinterpret_cast<const f32x4*>(&now.affine[2][at]), vz = *reinterpret_cast<const f32x4*>(&now.affine[3][at]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        af.ks[u][i] = ks[i];
                        af.kz[u][i] = kz[i];
                        af.vs[u][i] = vs[i];
                        af.vz[u][i] = vz[i];
                    }
                }
                // V's operands are on their way while the probabilities are made
                constexpr int AHEAD = Sh::NT < 8 ? Sh::NT : 8;
                bf16x8 v[AHEAD], p[R];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) v[i] = __builtin_bit_cast(bf16x8, now.v[g][i][lane]);
                probabilities<D, R>(st, p, s, af, w.zq, sg);
                count_middle<D, BITS, R>(st, p);
#pragma unroll
                for (int i = 0; i < Sh::NT; ++i) {
                    const bf16x8 x = i < AHEAD ? v[i < AHEAD ? i : 0] : __builtin_bit_cast(bf16x8, now.v[g][i][lane]);
#pragma unroll
                    for (int r = 0; r < R; ++r) st.o[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, p[r], st.o[r][i], 0, 0, 0);
                }
            }
            __syncthreads();
            if constexpr (SETS == 1) {
                prepare_next();
                __syncthreads();
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float l = sum_over_quads(st.l[r]);
        const float z = fmaf(st.c[r][0], -0x1p29f, sum_over_quads(st.z[r]));
        if (!w.real[r]) continue;
        if (a.splits == 1) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            __bf16* o = static_cast<__bf16*>(a.o) + (int64_t)w.out[r] * D;
            each_run<D, BITS, R>(st, r, z, [&](int d, auto& v) {
                constexpr int N = sizeof(v) / 4;
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] *= inv;
                store_bf16<N>(o + d, v);
            });
        } else {
            const int64_t at = (int64_t)sh.split * a.batch * a.T * a.H + w.out[r];
            if (t_begin < t_end)
                each_run<D, BITS, R>(st, r, z, [&](int d, auto& v) {
                    constexpr int N = sizeof(v) / 4;
#pragma unroll
                    for (int k = 0; k < N; ++k) a.part_o[at * D + d + k] = v[k];
                });
            if (qd == 0) {
                a.part_ml[at * 2] = st.m[r];
                a.part_ml[at * 2 + 1] = l;
            }
        }
    }
}

// The parts of a split sequence together: a wave a query row, 4 elements a lane at a time.
__global__ __launch_bounds__(256) void kv_attend_join_kernel(CacheArgs a) {
    const int64_t rows = (int64_t)a.batch * a.T * a.H;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= rows) return;
    float m = kLowest, l = 0.0f;
    if (lane < a.splits) {
        m = a.part_ml[(lane * rows + row) * 2];
        l = a.part_ml[(lane * rows + row) * 2 + 1];
    }
    float top = m;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
    const float w = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - top);
    const float sum = wave_sum(l == 0.0f ? 0.0f : w * l);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    // heads of up to 256: 4 elements a lane. Lanes past a smaller head stay in the loop, as
    // their weights are read from it (they add up element 0 and store nothing).
    const int d = lane * 4 < a.hd ? lane * 4 : 0;
    f32x4 v = {0, 0, 0, 0};
    for (int s0 = 0; s0 < a.splits; s0 += 4) {   // 4 loads in flight
        f32x4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t s = min(s0 + k, a.splits - 1);
            x[k] = *reinterpret_cast<const f32x4*>(a.part_o + (s * rows + row) * a.hd + d);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float ws = s0 + k < a.splits ? __shfl(w, s0 + k) : 0.0f;
            // an empty part's values were never written
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(ws, ws == 0.0f ? 0.0f : x[k][e], v[e]);
        }
    }
    const float o[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
    if (lane * 4 < a.hd) store_bf16<4>(static_cast<__bf16*>(a.o) + row * a.hd + d, o);
}

// Rows of a wave of the chunk kernel (in tiles of 16), and sets of operands (of 64 (4 D + 16)
// bytes each): as two workgroups a CU leave registers and LDS (8 bits with heads of 128 spill
// 40 bytes a lane).
constexpr int kChunkWaves = 4;
constexpr int chunk_tiles(int64_t d) { return d <= 128 ? 2 : 1; }
constexpr int chunk_sets(int64_t d) { return d <= 128 ? 2 : 1; }

template <int D, int BITS>
void launch_shape(const fp::AttendPlan& p, const CacheArgs& a, unsigned grid, hipStream_t st) {
    if (p.chunk)
        hipLaunchKernelGGL((kv_attend_chunk_kernel<D, BITS, chunk_tiles(D), kChunkWaves, chunk_sets(D)>), dim3(grid),
                           dim3(kChunkWaves * 64), 0, st, a);
    else if (D > 128 || p.row_tiles == 1)
        hipLaunchKernelGGL((kv_attend_kernel<D, BITS, 1>), dim3(grid), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((kv_attend_kernel<D, BITS, D <= 128 ? 2 : 1>), dim3(grid), dim3(256), 0, st, a);
}

}  // namespace

namespace fp {

bool plan_attend(const kv_cache_desc& d, int64_t kvh, AttendPlan* out) {
    const int64_t hd = d.head_dim;
    if (hd != 32 && hd != 64 && hd != 96 && hd != 128 && hd != 192 && hd != 256) return false;
    const int64_t rows = d.n_heads / kvh * d.tokens, heads = d.batch * kvh > 0 ? d.batch * kvh : 1;
    AttendPlan p;
    p.chunk = rows > 32;
    p.row_tiles = rows <= 16 || hd > 128 ? 1 : 2;   // two tiles of a wider head would spill
    const int64_t block = 16 * (p.chunk ? chunk_tiles(hd) * kChunkWaves : p.row_tiles);
    p.row_blocks = (int32_t)((rows + block - 1) / block);
    // Parts of a sequence, equal ones whatever its length (which the device alone knows):
    // enough workgroups to fill the card, with parts long enough to be worth their queries and
    // their join. Parts of one size for all sequences measured slower (104 us instead of 84
    // for 64 sequences of 2500 to 8191 positions). Few rows: half as many workgroups again
    // where parts are longer than 2048 positions (63 sequences up to 8191: 2 parts 83 us, 3 parts
    // 79), not where they are shorter (24 of up to 3333: 4 parts 22.5 us, 6 parts 23.2). The
    // rule does not count the workgroups that are resident, three a CU for both: 768, of which
    // these are 1.3 and 2.0, 1.5 and 2.25 rounds.
    const int64_t positions = d.max_pages * d.page_size, least = p.chunk ? 512 : 256;
    const auto parts = [&](int64_t want) { return (want + heads * p.row_blocks - 1) / (heads * p.row_blocks); };
    const int64_t want = p.chunk ? 512 : positions > 2048 * parts(1024) ? 1536 : 1024;
    int64_t splits = parts(want);
    if (p.chunk && 4 * heads * p.row_blocks > 3 * want) splits = 1;
    if (splits > (positions + least - 1) / least) splits = (positions + least - 1) / least;
    p.splits = (int32_t)(splits < 1 ? 1 : splits > 64 ? 64 : splits);
    if (heads * p.row_blocks * p.splits > (int64_t(1) << 23)) return false;   // of 256 threads: one grid
    if (p.splits > 1) p.workspace = (size_t)p.splits * (size_t)(d.batch * d.tokens * d.n_heads) * (size_t)(hd + 2) * 4;
    *out = p;
    return true;
}

hipError_t launch_attend(const kv_cache_desc& d, const AttendPlan& p, const CacheArgs& a, hipStream_t st) {
    const unsigned grid = (unsigned)((int64_t)a.batch * a.KVH * p.row_blocks * p.splits);
#define KV_CASE(D)                                       \
    if (d.head_dim == D) {                               \
        if (d.bits == 4)                                 \
            launch_shape<D, 4>(p, a, grid, st);          \
        else                                             \
            launch_shape<D, 8>(p, a, grid, st);          \
    }
    KV_CASE(32) KV_CASE(64) KV_CASE(96) KV_CASE(128) KV_CASE(192) KV_CASE(256)
#undef KV_CASE
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.splits > 1) {
        const int64_t rows = (int64_t)a.batch * a.T * a.H;
        hipLaunchKernelGGL(kv_attend_join_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace fp
