// What the kernels of attention over whole prompts share (formulas, layouts and the meaning of
// every size are in include/prompt_attention.h).
//
// Tiles. One operand of a workgroup's products stays in registers (a wave's 32 rows), the
// other passes through LDS in tiles of rows, two tensors at a time (k and v, or q and do),
// fetched by direct-to-LDS loads one tile ahead. A first product X = A B^T (A the tile's rows,
// B the wave's) leaves a lane 16 of 32 tile rows of one of the wave's rows - row lane % 32 -
// and those 16, rounded to bf16, are an operand of the second product Y^T = A'^T X as they lie,
// if the tile's rows are counted as the lanes hold them: 4 (lane / 32) + 8 (i / 4) + i % 4.
// Nothing is exchanged between lanes but row maxima and sums. A' is read from LDS transposed.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/prompt_attention.h"
#include "device_common.h"
#include "fused_proj_kernels.h"

namespace fp {

struct AttentionArgs {
    const char *q, *k, *v, *d_o;
    const __bf16* o_in;
    const int32_t* extents;
    __bf16* o;
    float* lse;                  // [b*H, T], forward: or nullptr
    const float* lse_in;
    __bf16 *dq, *dk, *dv;
    float* stats;                // backward: [b*H, T] lse log2(e), then [b*H, T] D
    float* partial;              // backward: [kv_parts][dk, dv][b, KVH, T, hd], where kv_parts > 1
    int32_t part_heads;          // heads of a group that a workgroup of keys passes over
    int64_t q_sb, q_sh, k_sb, k_sh, v_sb, v_sh;   // bytes
    uint32_t q_st, k_st, v_st, o_st;              // bytes between tokens
    int32_t batch, T, H, KVH, hd, group, sequences, causal;
    int32_t tiles;               // workgroups over a head's tokens
    uint32_t blocks;
    float scale, scale_log2;     // sm_scale, sm_scale log2(e)
    FastDivU31 div_tiles, div_group, div_kvh;
};

struct AttentionPlan {
    int32_t dim = 0;             // the kernels' head size, hd or the next one that is compiled
    int64_t rows = 0;            // b T H
    int32_t kv_parts = 1;        // parts that a group's heads are cut into for dk and dv
    size_t backward_workspace = 0;
};

// Whether workgroups of 128 tokens (4 waves, two workgroups a CU) are so few, or with a causal mask so different, that
// workgroups of 64 with 4 waves a row are faster. Forward pass, heads of 64 and 128, us, workgroups of 128 / of 64:
//   8 heads x 2048 tokens (128 workgroups)  37 / 20, 52 / 31      the same, causal  37 / 20, 52 / 29
//   64 x 512 (256)                          13 / 13, 18 / 24      16 x 2048, causal (256)  38 / 29, 52 / 38
//   128 x 512 (512)                         17 / 22, 30 / 47      16 x 4096, causal (512)  89 / 65, 132 / 121
//   32 x 2048 (512)                         51 / 59, 83 / 114     64 x 2048, causal (1024) 74 / 75, 122 / 141
// Up to 128 tokens there are one or two tiles of keys, and nothing to share. Large groups gain less: 32 heads on 8 of 128 x 2048,
// causal (512) take 57 / 71, so the border for causal heads of 128 is drawn between them and 16 ungrouped heads x 4096, which
// lose by it (132 / 121).
inline bool few_workgroups(int64_t blocks, const prompt_attention_desc& d) {
    return d.tokens > 128 && (blocks < 256 || (d.tokens >= 1024 && blocks < (d.causal && d.head_dim <= 64 ? 768 : 512)));
}

// Sequences of up to 64 tokens: workgroups with a row of waves for every 32 that there are, and none idle. Forward and
// backward, us, 128 tokens a workgroup / these: 512 x 32 tokens, 32 heads on 8 of 128, causal, 156, 439 / 95, 260; 512 x 17, 12
// of 64, 24, 83 / 14, 40; 256 x 64, 32 on 8 of 128, 96, 304 / 83, 277. One sequence of 64 has no gain (backward 26 / 34).
inline int short_rows(const prompt_attention_desc& d) {   // 0: the sequences are not short
    if (d.tokens <= 32) return 1;
    return d.tokens <= 64 && d.batch * d.n_heads >= 512 ? 2 : 0;
}

// Sets kv_parts.
void plan_attention_backward(const prompt_attention_desc& d, int64_t kvh, AttentionPlan* p);
hipError_t launch_attention(const prompt_attention_desc& d, const AttentionPlan& p, AttentionArgs a, hipStream_t st);
hipError_t launch_attention_backward(const prompt_attention_desc& d, const AttentionPlan& p, AttentionArgs a, hipStream_t st);

namespace dev {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

// A workgroup's place: which tile of tokens of which head. Workgroups go round-robin to the 8
// XCDs; each XCD takes consecutive ones of the order (batch row, k/v head, tile, head of the
// group), so that those which read the same k and v share an L2.
struct Place {
    int32_t batch, head, kvh, tile;
};
__device__ __forceinline__ uint32_t in_xcd_order(uint32_t block, uint32_t blocks) {
    const uint32_t xcd = block & 7, q = blocks >> 3, r = blocks & 7;
    return xcd * q + (xcd < r ? xcd : r) + (block >> 3);
}

// Which rows of the other side a token sees: first .. last; none where first is kNone (then last is it, too).
struct Span {
    int32_t first, last;
};
constexpr int32_t kNone = 0x7FFFFFFF;
__device__ __forceinline__ bool sees(Span s, int at) { return (uint32_t)(at - s.first) <= (uint32_t)(s.last - s.first); }

// The same value in every lane: `f` over all 64 lanes' x (f associative and commutative).
template <typename F>
__device__ __forceinline__ int32_t over_lanes(int32_t x, F f) {
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true));    // quads: lane ^ 1
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true));    // lane ^ 2
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true));   // half rows mirrored
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0x128, 0xF, 0xF, true));   // rows rotated by 8
    auto r = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
    x = f((int32_t)r[0], (int32_t)r[1]);
    r = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)x, false, false);
    return __builtin_amdgcn_readfirstlane(f((int32_t)r[0], (int32_t)r[1]));
}

// The sequences of a workgroup's rows row0 .. row0 + BM - 1, and of this lane's row, one of the 32 of
// its wave from `mine0` on (lane % 32): [first, last] tokens.
struct Spans {
    Span mine;            // first kNone: of no sequence
    Span first, last;     // of the first and the last row of the workgroup that is of one
    int32_t from, to;     // these rows (from > to: none)
};
// Every wave for itself, without LDS: an offset a lane, 64 at a time. starts, ends: which of the two are
// wanted (reductions over the lanes are what it takes most of its time for).
template <int BM>
__device__ __forceinline__ Spans find_spans(const AttentionArgs& a, int batch, int row0, int mine0, bool starts, bool ends) {
    const int lane = threadIdx.x & 63, mine = mine0 + (lane & 31);
    Spans s;
    if (a.sequences == 0) {
        int length = a.T;
        if (a.extents) length = __builtin_amdgcn_readfirstlane(min(max(a.extents[batch], 0), a.T));
        s.from = row0;
        s.to = min(row0 + BM, length) - 1;
        s.first = s.last = Span{0, length - 1};
        s.mine = mine < length ? s.first : Span{kNone, kNone};
        return s;
    }
    const auto greatest = [](int32_t x, int32_t y) { return max(x, y); };
    const auto least = [](int32_t x, int32_t y) { return min(x, y); };
    const auto either = [](int32_t x, int32_t y) { return x | y; };
    const int32_t begin = a.extents[0], end = a.extents[a.sequences];
    int32_t at = lane <= a.sequences ? a.extents[lane] : 0;
    const int first = __builtin_amdgcn_readfirstlane(min(max(begin, 0), a.T)), behind = __builtin_amdgcn_readfirstlane(min(max(end, 0), a.T));
    s.from = max(row0, first);
    s.to = min(row0 + BM, behind) - 1;
    // the greatest offsets not above, and the least above, of the workgroup's first and last row and
    // the wave's 32; those between the wave's rows as bits
    int32_t a0 = 0, a1 = a.T, b0 = 0, b1 = a.T, m0 = 0, m1 = a.T, bits = 0;
    for (int i = 0; i <= a.sequences; i += 64) {
        if (i > 0) at = i + lane <= a.sequences ? a.extents[i + lane] : 0;
        const bool is = i + lane <= a.sequences;
        at = min(max(at, 0), a.T);
        const auto below = [&](int32_t& x, int32_t& y, int32_t r) {
            if (is && at <= r) x = max(x, at);
            if (is && at > r) y = min(y, at);
        };
        below(a0, a1, s.from);
        below(b0, b1, s.to);
        if (is && at <= mine0) m0 = max(m0, at);
        if (is && at >= mine0 + 32) m1 = min(m1, at);
        if (is && at > mine0 && at < mine0 + 32) bits |= (int32_t)(1u << (at - mine0));
    }
    if (starts) {
        a0 = over_lanes(a0, greatest);
        b0 = over_lanes(b0, greatest);
        m0 = over_lanes(m0, greatest);
    }
    if (ends) {
        a1 = over_lanes(a1, least);
        b1 = over_lanes(b1, least);
        m1 = over_lanes(m1, least);
    }
    s.first = Span{a0, a1 - 1};
    s.last = Span{b0, b1 - 1};
    const uint32_t cuts = (uint32_t)over_lanes(bits, either);
    const uint32_t below = cuts & (~0u >> (31 - (lane & 31))), above = cuts & ~(~0u >> (31 - (lane & 31)));
    s.mine = Span{below ? mine0 + 31 - __clz(below) : m0, (above ? mine0 + __ffs(above) - 1 : m1) - 1};
    if (mine < first || mine >= behind) s.mine = Span{kNone, kNone};
    return s;
}

// LDS rows of D elements in chunks of 16 bytes, the chunk index xored with f(row) inside groups of G
// (64 banks of 4 bytes hold 16 chunks): 16 rows read at one chunk, and 4 rows at two neighbouring
// ones (a transposing read), come from different banks.
template <int D>
struct Rows {
    static constexpr int CPR = D / 8, BYTES = D * 2;
    static constexpr int G = CPR % 16 == 0 ? 16 : CPR % 8 == 0 ? 8 : 4;
    static __device__ __forceinline__ int swizzle(int row) {
        if constexpr (G == 16) return ((row & 3) << 2) | ((row >> 2) & 3);
        if constexpr (G == 8) return ((row & 2) << 1) | ((row >> 2) & 3);
        return (row >> 2) & 3;
    }
    // Operand A of X: row lane % 32, elements 16 kk + 8 (lane / 32) .. + 7.
    static __device__ __forceinline__ unsigned plain_base() {
        const int lane = threadIdx.x & 63, row = lane & 31;
        return (unsigned)(row * BYTES + (((lane >> 5) ^ swizzle(row)) << 4));
    }
    static __device__ __forceinline__ bf16x8 plain(unsigned base, int row32, int kk) {
        const unsigned at = (base ^ (unsigned)(((2 * kk) % G) << 4)) + (2 * kk) / G * G * 16 + row32 * 32 * BYTES;
        return *(const __attribute__((address_space(3))) bf16x8*)(size_t)at;
    }
    // Operand A of Y^T: element 32 t + lane % 32 of rows 16 s + 4 (lane / 32) + {0 .. 3, 8 .. 11}.
    // part: of two, where a wave has every other tile of Y^T.
    static __device__ __forceinline__ unsigned turned_base(int part = 0) {
        const int lane = threadIdx.x & 63, g = lane >> 4, q = lane & 15;
        const int row = 4 * (g >> 1) + (q >> 2), chunk = 4 * part + (g & 1) * 2 + ((q & 3) >> 1);
        return (unsigned)(row * BYTES + ((chunk ^ swizzle(row)) << 4) + (q & 1) * 8);
    }
    static __device__ __forceinline__ i16x4 turned_half(unsigned base, int t, int s, int j) {
        const unsigned at = (base ^ (unsigned)((((4 * t) % G) ^ (2 * j)) << 4)) + (4 * t) / G * G * 16 + (16 * s + 8 * j) * BYTES;
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(size_t)at);
    }
    static __device__ __forceinline__ bf16x8 turned(unsigned base, int t, int s) {
        const i16x4 lo = turned_half(base, t, s, 0), hi = turned_half(base, t, s, 1);
        return __builtin_bit_cast(bf16x8, i16x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w});
    }
};

// The same address in SGPRs.
__device__ __forceinline__ const char* uniform(const char* p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<const char*>(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) << 32) |
                                         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a));
}

// Direct-to-LDS loads of a tile of BN rows of one tensor, by NW waves. A lane's 16 bytes of
// instruction n land in LDS chunk 64 n + lane, so the source chunk is the one that belongs there.
// KEEP: the lanes' offsets stay in registers; else they are made again for every tile.
template <int D, int BN, int NW, bool PADDED, bool KEEP = true>
struct TileLoads {
    using R = Rows<D>;
    static constexpr int TOTAL = BN * R::CPR / 64, N = (TOTAL + NW - 1) / NW;
    static_assert(TOTAL * 64 == BN * R::CPR, "whole instructions");
    uint32_t offset[KEEP ? N : 1];
    static __device__ __forceinline__ int row_of(int i, int tid) { return (i * NW * 64 + tid) / R::CPR; }
    static __device__ __forceinline__ int chunk_of(int i, int tid) {
        const int slot = (i * NW * 64 + tid) % R::CPR;
        return slot / R::G * R::G + ((slot % R::G) ^ R::swizzle(row_of(i, tid)));
    }
    __device__ __forceinline__ void init(uint32_t stride) {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < N; ++i) offset[i] = (uint32_t)row_of(i, threadIdx.x) * stride + (uint32_t)chunk_of(i, threadIdx.x) * 16;
        }
    }
    // Rows from `from` on (wave-uniform) to LDS address `tile`; rows at or past `count` repeat the last one there is.
    __device__ __forceinline__ void issue(const char* from, uint32_t stride, unsigned tile, int count, int hd) const {
        int tid = threadIdx.x;
        if constexpr (!KEEP) asm volatile("" : "+v"(tid));   // what follows from it is not kept since the last tile
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const char* src = uniform(from);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (TOTAL % NW != 0 && i * NW + wave >= TOTAL) break;
            const int row = count >= BN ? row_of(i, tid) : min(row_of(i, tid), count - 1);
            const uint32_t at = KEEP && count >= BN ? offset[KEEP ? i : 0] : (uint32_t)row * stride + (uint32_t)chunk_of(i, tid) * 16;
            const unsigned dst = tile + (unsigned)(i * NW + wave) * 1024;
            // The wait states: a VMEM instruction that reads an SGPR which VALU wrote needs 5, a
            // direct-to-LDS load after a write of M0 1. Inline, so that the compiler does not wait
            // for the loads of the next tile before it reads this one.
            if (!PADDED || chunk_of(i, tid) * 8 < hd)
                asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(at), "s"(src), "{m0}"(dst) : "memory");
        }
    }
};
// All outstanding loads of this wave have landed, and its reads of LDS are done (a workgroup of one wave has no
// barrier that waits for them).
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }
// This wave's writes to LDS are done, before direct-to-LDS loads to the same place, which come by another path. The barrier behind
// it does not see to that in a workgroup of one wave, where it is none.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// 32 rows of a wave as operand B of X: row lane % 32 of `src` rows (64-bit address of the lane's
// row), elements 16 kk + 8 (lane / 32) .. + 7; zeros behind hd and for rows that are not there.
template <int D>
__device__ __forceinline__ void load_rows(bf16x8 (&to)[D / 16], const char* row, bool there, int hd) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        u32x4 x = {0, 0, 0, 0};
        if (there && 16 * kk + 8 * h < hd) x = *reinterpret_cast<const u32x4*>(row + 32 * kk + 16 * h);
        to[kk] = __builtin_bit_cast(bf16x8, x);
    }
}

// Makes the compiler wait here for operands that it loads. It would wait at their first use, inside the
// loop over the tiles, in every round, and with it for the tile that is on its way.
template <int N>
__device__ __forceinline__ void arrived(bf16x8 (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        u32x4 w = __builtin_bit_cast(u32x4, x[i]);
        asm volatile("" : "+v"(w));
        x[i] = __builtin_bit_cast(bf16x8, w);
    }
}

// The rows of a lane's 16 values of a 32 x 32 product.
__device__ __forceinline__ int value_row(int i) { return (i & 3) + 8 * (i >> 2) + 4 * ((threadIdx.x & 63) >> 5); }

// X, rounded, as operands B of Y^T. Probabilities are one bf16 number: o and dv are off by 0.0023 of their norm then, of which 0.0017 is
// their own rounding. As two numbers, a product more, they would be off by that alone, and 8192 tokens, 32 heads on 8 of 128, causal,
// would take 762 us for 573, forward and backward of 2 x 4096 1746 for 1553, of a ragged batch of 32 x 512, 12 of 64, 160 for 145.
template <int NB>
__device__ __forceinline__ void to_operands(bf16x8 (&o)[2 * NB], const f32x16 (&x)[NB]) {
#pragma unroll
    for (int s = 0; s < 2 * NB; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[s][i] = (__bf16)x[s >> 1][8 * (s & 1) + i];
}

// bf16 pairs whose exponent is the largest (infinities and NaN) as masks of 16 bits.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    const uint32_t up = (w & 0x7F807F80u) + 0x00800080u;   // bit 15 of a half: its exponent was 255
    return ((up >> 15) & 0x00010001u) * 0xFFFFu;
}
__device__ __forceinline__ bf16x8 only_finite(bf16x8 x) {
    u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= ~not_finite(w[i]);
    return __builtin_bit_cast(bf16x8, w);
}

// X = A B^T for NB blocks of 32 rows of the tile whose plain base is given; b(kk): operand B. Operands are read ahead of
// their products, in groups (of J steps) that the compiler keeps apart: it would read them all at
// once else, into registers that there are not.
template <int D, int NB, int J, typename B>
__device__ __forceinline__ void product(f32x16 (&x)[NB], const B& b, unsigned base) {
    using R = Rows<D>;
    constexpr int K = D / 16;
    bf16x8 a[2][J][NB], w[2][J];
    const auto read = [&](int k) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            w[k / J % 2][j] = b(k + j);
#pragma unroll
            for (int u = 0; u < NB; ++u) a[k / J % 2][j][u] = R::plain(base, u, k + j);
        }
    };
#pragma unroll
    for (int u = 0; u < NB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[u][i] = 0.0f;
    read(0);
#pragma unroll
    for (int k = 0; k < K; k += J) {
        if (k + J < K) read(k + J);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int u = 0; u < NB; ++u)
                x[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[k / J % 2][j][u], w[k / J % 2][j], x[u], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// What that rounding leaves, rounded: the two together have 16 bits of X.
template <int NB>
__device__ __forceinline__ void rest_to_operands(bf16x8 (&o)[2 * NB], const bf16x8 (&first)[2 * NB], const f32x16 (&x)[NB]) {
#pragma unroll
    for (int s = 0; s < 2 * NB; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[s][i] = (__bf16)(x[s >> 1][8 * (s & 1) + i] - (float)first[s][i]);
}

// Y^T += A'^T X for the tile of 32 NB rows whose turned base is given; C tiles of Y^T a group. PARTS: the wave has every
// PARTS-th tile (32 elements of the heads) of Y^T alone, the first as turned_base says. rest: of X, the same way.
// Where the mask hides some of the tile's rows from some of the wave's (`edge`), their values in X
// are 0, but 0 times an infinity or NaN is NaN. A product of the tile with zeros tells whether it
// holds any; then they are left out here, and true is returned: add_left_out has to follow.
template <int D, int NB, int C, int PARTS = 1>
__device__ __forceinline__ bool add_turned(f32x16 (&y)[D / 32 / PARTS], const bf16x8 (&x)[2 * NB], unsigned base, bool edge,
                                           const bf16x8* rest = nullptr) {
    using R = Rows<D>;
    constexpr int T = D / 32 / PARTS, S = 2 * NB, P = T / C;   // P groups a step
    static_assert(P * C == T, "whole groups");
    bf16x8 a[2][C];
    const auto read = [&](int i) {
#pragma unroll
        for (int c = 0; c < C; ++c) a[i & 1][c] = R::turned(base, (i % P * C + c) * PARTS, i / P);
    };
    bool all_finite = true;
    if (edge) {
        f32x4 probe = {0, 0, 0, 0};
        const bf16x8 zeros = {};
#pragma unroll
        for (int i = 0; i < S * P; ++i) {
            read(i);
#pragma unroll
            for (int c = 0; c < C; ++c) probe = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i & 1][c], zeros, probe, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // a NaN in a row of A makes the product's whole row NaN: each lane has 4 of its rows
        all_finite = !__any(probe[0] != 0.0f || probe[1] != 0.0f || probe[2] != 0.0f || probe[3] != 0.0f);
    }
    read(0);
#pragma unroll
    for (int i = 0; i < S * P; ++i) {
        if (i + 1 < S * P) read(i + 1);
        if (!all_finite) {
            asm volatile("");   // a branch, not selects
#pragma unroll
            for (int c = 0; c < C; ++c) a[i & 1][c] = only_finite(a[i & 1][c]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            y[i % P * C + c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i & 1][c], x[i / P], y[i % P * C + c], 0, 0, 0);
        if (rest) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                y[i % P * C + c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i & 1][c], rest[i / P], y[i % P * C + c], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    return !all_finite;
}

// What add_turned left out of the tiles of BN rows from `low` on, up to row `high`: their infinities and
// NaN (as NaN, with AS_NAN), straight from memory, added to the rows that see them. `rows`: row 0; `edge(p)`: whether tile p was
// one. Behind the loop over the tiles, and not in it, where it would cost every wave registers.
template <int D, int BN, bool AS_NAN, int PARTS = 1, typename Edge>
__device__ __forceinline__ void add_left_out(f32x16 (&y)[D / 32 / PARTS], const char* rows, uint32_t stride, int low, int high,
                                             Span mine, int hd, Edge edge, int part = 0) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll 1
    for (int p = low; p <= high; p += BN) {
        if (!edge(p)) continue;
#pragma unroll 1
        for (int row = p; row < p + BN && row <= high; ++row) {
            const bool see = sees(mine, row);
#pragma unroll
            for (int i = 0; i < D / 8 / PARTS; ++i) {
                const int d = 32 * ((i >> 2) * PARTS + part) + 8 * (i & 3);
                u32x2 e = {0, 0};
                if (d < hd) e = *reinterpret_cast<const u32x2*>(rows + (int64_t)row * stride + 2 * d + 8 * h);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t bits = k & 1 ? e[k >> 1] & 0xFFFF0000u : e[k >> 1] << 16;
                    if (see && (bits & 0x7F800000u) == 0x7F800000u) y[i >> 2][4 * (i & 3) + k] += __uint_as_float(AS_NAN ? 0x7FC00000u : bits);
                }
            }
        }
    }
}

// Y^T times `by` as bf16, each lane's row of it to its `to`, elements below hd: a lane and the one
// 32 further exchange halves, so that each stores 16 bytes.
template <int D, int PARTS = 1>
__device__ __forceinline__ void store_turned(__bf16* to, const f32x16 (&y)[D / 32 / PARTS], float by, int hd, int part = 0) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int t = 0; t < D / 32 / PARTS; ++t)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            bf16x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = (__bf16)(y[t][8 * p + i] * by);
                b[i] = (__bf16)(y[t][8 * p + 4 + i] * by);
            }
            const u32x2 wa = __builtin_bit_cast(u32x2, a), wb = __builtin_bit_cast(u32x2, b);
            u32x4 out;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto r = __builtin_amdgcn_permlane32_swap(wa[i], wb[i], false, false);
                out[i] = r[0];
                out[2 + i] = r[1];
            }
            const int d = 32 * (t * PARTS + part) + 16 * p + 8 * h;
            if (d < hd) *reinterpret_cast<u32x4*>(to + d) = out;
        }
}

// Sums of the H waves of each of RW rows of waves into wave `taker` of the row (turn: which one this is), through `memory`
// (16-byte aligned LDS of (H - 1) RW 128 D bytes, which other waves may still read).
template <int D, int RW, int H>
__device__ __forceinline__ void sum_up(f32x16 (&y)[D / 32], int taker, int wave, int turn, unsigned char* memory) {
    constexpr int NEXT = RW * D * 8;   // from one wave of a row to its next, in pieces of 16 bytes
    f32x4* const shared = reinterpret_cast<f32x4*>(memory) + wave * D * 8 + (threadIdx.x & 63);
    __syncthreads();
    if (turn != taker) {
        f32x4* const to = shared + (turn > taker ? turn - 1 : turn) * NEXT;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
            to[j * 64] = f32x4{y[j >> 2][4 * (j & 3)], y[j >> 2][4 * (j & 3) + 1], y[j >> 2][4 * (j & 3) + 2], y[j >> 2][4 * (j & 3) + 3]};
    }
    __syncthreads();
    if (turn == taker) {
#pragma unroll
        for (int g = 0; g < H - 1; ++g)
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                const f32x4 x = shared[g * NEXT + j * 64];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[j >> 2][4 * (j & 3) + i] += x[i];
            }
    }
}

// The first row of a wave's 32 that is of a sequence, the last one, and what all of them, and any of
// them, see (spans go up with the rows).
struct WaveSight {
    bool any;
    int32_t low, high;             // some row sees low .. high
    int32_t full_from, full_to;    // every row (of a sequence) sees these
};
__device__ __forceinline__ WaveSight wave_sight(Span s) {
    WaveSight w;
    const uint32_t there = (uint32_t)__ballot(s.first != kNone);   // rows repeat in the upper lanes
    w.any = there != 0;
    const int a = there ? __ffs(there) - 1 : 0, b = there ? 31 - __clz(there) : 0;
    w.low = __builtin_amdgcn_readlane(s.first, a);
    w.full_from = __builtin_amdgcn_readlane(s.first, b);
    w.full_to = __builtin_amdgcn_readlane(s.last, a);
    w.high = __builtin_amdgcn_readlane(s.last, b);
    return w;
}

// From the least first to the greatest last row of NW waves' spans (each the same in all lanes of its wave).
template <int NW>
__device__ __forceinline__ Span of_workgroup(Span s) {
    if constexpr (NW > 1) {
        __shared__ Span spans[NW];
        if ((threadIdx.x & 63) == 0) spans[threadIdx.x >> 6] = s;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NW; ++i) s = Span{min(s.first, spans[i].first), max(s.last, spans[i].last)};
    }
    return Span{__builtin_amdgcn_readfirstlane(s.first), __builtin_amdgcn_readfirstlane(s.last)};
}

}  // namespace dev
}  // namespace fp
