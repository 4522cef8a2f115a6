// Attention over the key/value cache in 4 or 8 bits (gfx950; formulas and format are in
// include/kv_cache.h), on the bf16 matrix cores without dequantising.
//
// Codes as bf16 numbers. The bf16 number with the bits of a code c (0..255) is c 2^-133: the
// 7 mantissa bits of a denormal and the lowest exponent bit go on linearly, and the matrix
// cores take denormal inputs as they are. So a code becomes an operand by masking alone,
// and its products with q are exact. With 4 bits, every other code is masked where it lies,
// 4 bits up, and stands for 16 c 2^-133: those elements of q are divided by 16, those of the
// output at the end. q is multiplied by the power of two that brings the wave's largest
// value to 2^100, so that the products are ordinary numbers.
//
// The affine format stays outside the products. With a token's scale s and zero z,
//   q . khat = s (q . c) + z sum(q)
//   sum_j p_j vhat_j = sum_j b_j (c_j - C) + sum_j p_j (z_j + C s_j),    b_j = p_j s_j in bf16
// C is the middle code: codes are positive, so the rounding of b_j times c_j would be that of
// a sum far larger than the result; times c_j - C it is the rounding of the values' own
// spread (measured: output error 0.0021 of the output's norm instead of 0.0049, of which
// 0.0017 is the output's own rounding). C sum_j b_j is one more product, with a constant.
//
// Tiles. A wave holds R x 16 query rows (all rows of a k/v head: token by token, its group's
// heads inside) and takes 32 positions at a time, two halves of 16 that each lie in one
// page. S = K Q^T (16 positions x 16 rows a product) leaves each lane 4 positions of one
// row, which is the operand layout of O^T = V^T P^T if the 32 positions of that product are
// counted as the lanes hold them: nothing is exchanged between lanes but row maxima. K's
// operand is contiguous in memory up to a permutation of the head's elements, which q's
// operand shares. V's operand needs 8 positions of one element in a lane: a lane reads the
// same few bytes of 8 positions and pairs them up with byte permutes. Nothing goes through
// LDS, and waves do not wait for each other inside the loop.
#include <cmath>

#include "kv_cache.h"
#include "vector_io.h"

namespace {

using namespace fp::dev;
using fp::CacheArgs;

constexpr float kLowest = -3.0e38f;   // the running maximum before any position
constexpr float kLift = 80.0f;        // probabilities are held times 2^80: with a scale of at most 2^24 and
                                      // codes of 2^-133 their products neither overflow nor vanish
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

template <int D, int BITS>
__device__ __forceinline__ void load_tile(Tile<D, BITS>& t, const CacheArgs& a, const int32_t* table, int kvh, int tile,
                                          int length) {
    using Sh = Shape<D, BITS>;
    const int lane = threadIdx.x & 63, m = lane & 15, qd = lane >> 4;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int p = tile * 32 + u * 16;
        int64_t row = 0;   // any row that exists stands in for one that does not
        t.known[u] = 0;
        if (p < length) {
            const int pg = (int)fp::fastdiv_u31((uint32_t)p, a.div_page);
            const int page = __builtin_amdgcn_readfirstlane(table[pg]);
            if (page >= 0 && page < a.n_pages) {
                row = (int64_t)page * a.page_rows + (int64_t)kvh * a.page_size + (p - pg * a.page_size);
                t.known[u] = length - p < 16 ? length - p : 16;
            }
        }
        const uint8_t* kc = a.k_codes + row * Sh::ROWB;
        const uint8_t* vc = a.v_codes + row * Sh::ROWB;
        load_bytes<Sh::KW * 4>(t.k[u], kc + (m * Sh::ROWB + qd * (Sh::ROWB / 4)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            load_bytes<Sh::B0>(t.v0[u][j], vc + ((qd * 4 + j) * Sh::ROWB + m * Sh::B0));
            if constexpr (Sh::D1 > 0)
                load_bytes<Sh::B1>(t.v1[u][j], vc + ((qd * 4 + j) * Sh::ROWB + Sh::D0 * BITS / 8 + m * Sh::B1));
        }
        t.kp[u] = *reinterpret_cast<const u32x4*>(a.k_params + row + qd * 4);
        t.vp[u] = *reinterpret_cast<const u32x4*>(a.v_params + row + qd * 4);
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
    f32x4 o[R][D / 16];    // output tiles, in codes: see store order at finish()
    f32x4 c[R];               // 2 C sum_j b_j, in codes: the same in all four
    float m[R], l[R], z[R];   // running maximum (log2), and this lane's sums of p and of p (z + C s)
};

template <int D, int BITS, int R>
__device__ __forceinline__ void take_tile(State<D, R>& st, const Tile<D, BITS>& t, const bf16x8 (&q)[R][D / 32],
                                          const float (&zq)[R], const int (&last)[R], int first_last, float c1, int tile) {
    using Sh = Shape<D, BITS>;
    const int qd = (threadIdx.x & 63) >> 4;
    // whether any of the wave's rows does not see any of the 32 positions
    const bool edge = t.known[0] < 16 || t.known[1] < 16 || tile * 32 + 31 > first_last;
    float ks[2][4], kz[2][4], vs[2][4], vz[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ks[u][i] = param_scale(t.kp[u][i]) * c1;
            kz[u][i] = param_zero(t.kp[u][i]);
            vs[u][i] = param_scale(t.vp[u][i]);
            vz[u][i] = fmaf(vs[u][i], 0.5f * (float)((1 << BITS) - 1), param_zero(t.vp[u][i]));
        }
    bf16x8 p[R];
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
#pragma unroll
    for (int r = 0; r < R; ++r) {
        bool seen[2][4];
        if (edge) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = qd * 4 + i;
                    seen[u][i] = at < t.known[u] && tile * 32 + u * 16 + at <= last[r];
                }
        }
        float y[2][4];
        float top = -INFINITY;
        const float base = kLift - st.m[r];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[u][i] = fmaf(ks[u][i], s[r][u][i], fmaf(kz[u][i], zq[r], base));
                if (edge) y[u][i] = seen[u][i] ? y[u][i] : -INFINITY;
                top = fmaxf(top, y[u][i]);
            }
        if (__any(top > kLift + kSlack)) {
            // the maximum moves: the logits again, without the old one
            top = kLowest;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[u][i] = fmaf(ks[u][i], s[r][u][i], kz[u][i] * zq[r]);
                    if (edge) y[u][i] = seen[u][i] ? y[u][i] : -INFINITY;
                    top = fmaxf(top, y[u][i]);
                }
            const float m = fmaxf(st.m[r], max_over_quads(top));
            const float down = __builtin_amdgcn_exp2f(st.m[r] - m);
            st.m[r] = m;
            st.l[r] *= down;
            st.z[r] *= down;
#pragma unroll
            for (int i = 0; i < Sh::NT; ++i) st.o[r][i] *= down;
            st.c[r] *= down;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[u][i] = (y[u][i] - m) + kLift;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = __builtin_amdgcn_exp2f(y[u][i]);
                st.l[r] += e;
                float es = e * vs[u][i], ez = vz[u][i];
                if (edge) {
                    // a slot that is not seen may hold anything
                    es = seen[u][i] ? es : 0.0f;
                    ez = seen[u][i] ? ez : 0.0f;
                }
                st.z[r] = fmaf(e, ez, st.z[r]);
                p[r][u * 4 + i] = (__bf16)es;
            }
    }
    constexpr uint32_t kTwiceC = ((1u << BITS) - 1) * 0x00010001u;
    const bf16x8 twice_c = __builtin_bit_cast(bf16x8, u32x4{kTwiceC, kTwiceC, kTwiceC, kTwiceC});
#pragma unroll
    for (int r = 0; r < R; ++r) st.c[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(twice_c, p[r], st.c[r], 0, 0, 0);
    // pairs of positions, byte by byte of the lane's part of their rows
    const auto part = [&](auto bytes, auto first, const auto& w) {
        constexpr int B = decltype(bytes)::value, T0 = decltype(first)::value;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            constexpr uint32_t kPick = 0x0C040C00u;   // {0, byte of the second, 0, byte of the first}
            const uint32_t sel = kPick + 0x00010001u * (b & 3);
            u32x4 x;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) x[u * 2 + h] = __builtin_amdgcn_perm(w[u][2 * h + 1][b >> 2], w[u][2 * h][b >> 2], sel);
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
// its row, the values still to be divided by the row's sum. The lift ends here: codes of 2^-133
// under probabilities of 2^80 come back by 2^53 (the 4-bit codes masked 4 bits up by 2^49).
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
            for (int k = 0; k < N; ++k) v[k] = fmaf(st.o[r][T0 + k][i], BITS == 4 && (k & 1) ? 0x1p49f : 0x1p53f, z);
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

// WT waves of the workgroup's four take different positions of the same rows; 4 / WT different
// rows.
template <int D, int BITS, int R, int WT>
__global__ __launch_bounds__(256) void kv_attend_kernel(CacheArgs a) {
    using Sh = Shape<D, BITS>;
    constexpr int WR = 4 / WT, ROWS = R * 16, PAD = D + 4;
    __shared__ float both[WT > 1 ? WT * 16 * PAD : 1];
    __shared__ float both_ml[WT > 1 ? WT * 16 * 2 : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, n = lane & 15, qd = lane >> 4;
    // k/v heads fastest: the workgroups of one share an XCD's L2 where their number is a
    // multiple of 8; the last rows, which see the most, first
    const int heads = a.batch * a.KVH;
    const int head = (int)(blockIdx.x % (uint32_t)heads), rest = (int)(blockIdx.x / (uint32_t)heads);
    const int split = (int)fp::fastdiv_u31((uint32_t)rest, a.div_blocks);
    const int block = a.row_blocks - 1 - (rest - split * a.row_blocks);
    const int seq = (int)fp::fastdiv_u31((uint32_t)head, a.div_kvh), kvh = head - seq * a.KVH;
    const fp::Step step = fp::step_of(a, seq);
    const int rows = a.group * a.T;
    const int row0 = (block * WR + wave / WT) * ROWS;

    // the wave's rows: token of the step, head, position (-1: sees nothing)
    int last[R], row_out[R];
    bool real[R];
    const __bf16* qrow[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * 16 + n;
        real[r] = row < rows;
        const int s = real[r] ? (int)fp::fastdiv_u31((uint32_t)row, a.div_group) : 0, h = real[r] ? row - s * a.group : 0;
        last[r] = real[r] && s < step.count ? step.first + s : -1;
        const int qh = kvh * a.group + h;
        qrow[r] = static_cast<const __bf16*>(a.q) + ((int64_t)(seq * a.H + qh) * a.T + s) * D;
        row_out[r] = (seq * a.T + s) * a.H + qh;   // b T H fits 31 bits
    }
    // the positions that its first and its last real row see: rows are token by token
    const int s_first = (int)fp::fastdiv_u31((uint32_t)(row0 < rows ? row0 : 0), a.div_group);
    const int row_end = min(row0 + ROWS, rows) - 1;
    const int s_last = min((int)fp::fastdiv_u31((uint32_t)max(row_end, 0), a.div_group), step.count - 1);
    const bool any = row0 < rows && s_first < step.count;
    // rows that see nothing (padding) are masked by the edge path
    const int first_last = any && s_last * a.group + a.group - 1 >= row_end ? step.first + s_first : -1;
    const int sees = any ? max(min(step.length, step.first + s_last + 1), 0) : 0;
    const int tiles = (sees + 31) >> 5, per = (tiles + a.splits - 1) / a.splits;
    const int t_begin = split * per, t_end = min(tiles, t_begin + per);

    // q: exponents first
    u32x4 raw[R][Sh::KS];
    uint32_t top = 0;
    bool bad[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < Sh::KS; ++j) {
            raw[r][j] = last[r] >= 0 ? *reinterpret_cast<const u32x4*>(qrow[r] + qd * (D / 4) + j * 8) : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) mine = max(mine, max((raw[r][j][i] >> 7) & 0xFFu, (raw[r][j][i] >> 23) & 0xFFu));
        }
        mine = max(mine, (uint32_t)__shfl_xor((int)mine, 16));
        mine = max(mine, (uint32_t)__shfl_xor((int)mine, 32));
        bad[r] = mine >= 127 + 90;
        top = max(top, bad[r] ? 0u : mine);
    }
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, k));
    const int e = (int)max(top, 1u) - 127, lift = 100 - e;
    const float c1 = ldexpf(a.logit_scale, 133 - lift);
    bf16x8 q[R][Sh::KS];
    float zq[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < Sh::KS; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = bad[r] ? 0.0f : Piece<__bf16>::get(raw[r][j], operand_element<BITS>(i));
                sum += f;
                q[r][j][i] = (__bf16)ldexpf(f, BITS == 4 && (i & 2) ? lift - 4 : lift);   // exact
            }
        }
        sum = sum_over_quads(sum);
        zq[r] = bad[r] ? NAN : sum * a.logit_scale;
    }

    State<D, R> st;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        st.m[r] = kLowest;
        st.l[r] = st.z[r] = 0.0f;
        st.c[r] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < Sh::NT; ++i) st.o[r][i] = f32x4{0, 0, 0, 0};
    }
    const int32_t* table = a.table + (int64_t)seq * a.max_pages;
    for (int tile = t_begin + wave % WT; tile < t_end; tile += WT) {
        Tile<D, BITS> t;
        load_tile<D, BITS>(t, a, table, kvh, tile, step.length);
        take_tile<D, BITS, R>(st, t, q, zq, last, first_last, c1, tile);
    }

#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float l = sum_over_quads(st.l[r]) * 0x1p-80f, z = fmaf(st.c[r][0], -0x1p52f, sum_over_quads(st.z[r]) * 0x1p-80f);
        if constexpr (WT == 1) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            __bf16* o = static_cast<__bf16*>(a.o) + (int64_t)row_out[r] * D;
            if (real[r])
                each_run<D, BITS, R>(st, r, z, [&](int d, auto& v) {
                    constexpr int N = sizeof(v) / 4;
#pragma unroll
                    for (int k = 0; k < N; ++k) v[k] *= inv;
                    store_bf16<N>(o + d, v);
                });
        } else {
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
                const int s = (int)fp::fastdiv_u31((uint32_t)row, a.div_group), qh = kvh * a.group + row - s * a.group;
                const int64_t out = (int64_t)(seq * a.T + s) * a.H + qh;
                float m = kLowest, f[WT], sum = 0.0f, v[8];
#pragma unroll
                for (int w = 0; w < WT; ++w) m = fmaxf(m, both_ml[(w * 16 + rr) * 2]);
#pragma unroll
                for (int w = 0; w < WT; ++w) {
                    f[w] = __builtin_amdgcn_exp2f(both_ml[(w * 16 + rr) * 2] - m);
                    sum = fmaf(f[w], both_ml[(w * 16 + rr) * 2 + 1], sum);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    v[k] = 0.0f;
#pragma unroll
                    for (int w = 0; w < WT; ++w) v[k] = fmaf(f[w], both[(w * 16 + rr) * PAD + d + k], v[k]);
                }
                if (a.splits == 1) {
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] *= inv;
                    store_bf16<8>(static_cast<__bf16*>(a.o) + out * D + d, v);
                } else {
                    const int64_t at = (int64_t)split * a.batch * a.T * a.H + out;
                    f32x4* po = reinterpret_cast<f32x4*>(a.part_o + at * D + d);
                    po[0] = f32x4{v[0], v[1], v[2], v[3]};
                    po[1] = f32x4{v[4], v[5], v[6], v[7]};
                    if (d == 0) {
                        a.part_ml[at * 2] = m;
                        a.part_ml[at * 2 + 1] = sum;
                    }
                }
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
    for (int d = lane * 4; d < a.hd; d += 256) {
        f32x4 v = {0, 0, 0, 0};
        for (int s = 0; s < a.splits; ++s) {
            const float ws = __shfl(w, s);
            const f32x4 x = *reinterpret_cast<const f32x4*>(a.part_o + (s * rows + row) * a.hd + d);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = fmaf(ws, x[k], v[k]);
        }
        const float o[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
        store_bf16<4>(static_cast<__bf16*>(a.o) + row * a.hd + d, o);
    }
}

template <int D, int BITS>
void launch_shape(const fp::AttendPlan& p, const CacheArgs& a, unsigned grid, hipStream_t st) {
    constexpr int RL = D <= 128 ? 4 : 2;   // row tiles of a wave that registers hold
#define KV_CASE(R, WT)                                                                                \
    if (p.rows_per_wave == R && p.token_waves == WT) {                                                \
        hipLaunchKernelGGL((kv_attend_kernel<D, BITS, R, WT>), dim3(grid), dim3(256), 0, st, a);      \
        return;                                                                                       \
    }
    KV_CASE(1, 4)
    KV_CASE(2, 4)
    if constexpr (RL == 4) KV_CASE(4, 4)
    KV_CASE(RL, 1)
#undef KV_CASE
}

}  // namespace

namespace fp {

bool plan_attend(const kv_cache_desc& d, int64_t kvh, AttendPlan* out) {
    const int64_t hd = d.head_dim;
    if (hd != 32 && hd != 64 && hd != 96 && hd != 128 && hd != 192 && hd != 256) return false;
    const int64_t rows = d.n_heads / kvh * d.tokens, heads = d.batch * kvh;
    AttendPlan p;
    const int most = hd <= 128 ? 4 : 2;
    p.rows_per_wave = rows <= 16 ? 1 : rows <= 32 ? 2 : most;
    const int64_t wide = (rows + p.rows_per_wave * 64 - 1) / (p.rows_per_wave * 64);
    if (p.rows_per_wave == most && rows > 32 && heads * wide >= 256) {
        p.token_waves = 1;
        p.row_blocks = (int32_t)wide;
        p.splits = 1;
    } else {
        p.token_waves = 4;
        p.row_blocks = (int32_t)((rows + p.rows_per_wave * 16 - 1) / (p.rows_per_wave * 16));
        const int64_t tiles = (d.max_pages * d.page_size + 31) / 32;
        int64_t splits = heads > 0 ? (1024 + heads * p.row_blocks - 1) / (heads * p.row_blocks) : 1;
        if (splits > (tiles + 7) / 8) splits = (tiles + 7) / 8;
        if (splits > 64) splits = 64;
        p.splits = (int32_t)(splits < 1 ? 1 : splits);
    }
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
