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
    size_t run_workspace = 0, backward_workspace = 0;
};

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

// Which rows of the other side a token sees: first .. last; none where first is kNone.
struct Span {
    int32_t first, last;
};
constexpr int32_t kNone = 0x7FFFFFFF;

// LDS of find_spans.
template <int BM>
struct SpanMemory {
    int32_t start, after;
    uint32_t bits[BM / 32];
    Span of[BM];
};
// The sequences of tokens row0 .. row0 + BM - 1 into m.of, as [start, last token of the sequence]; returns the first and
// the last of these tokens that belong to any (first > last: none). All threads call it; ends with a barrier.
template <int BM>
__device__ __forceinline__ Span find_spans(SpanMemory<BM>& m, const AttentionArgs& a, int batch, int row0) {
    const int tid = threadIdx.x, row = row0 + tid;
    Span real;
    if (a.sequences == 0) {
        int length = a.T;
        if (a.extents) length = min(max(a.extents[batch], 0), a.T);
        real = Span{row0, min(row0 + BM, length) - 1};
        if (tid < BM) m.of[tid] = row < length ? Span{0, length - 1} : Span{kNone, kNone};
        __syncthreads();
        return real;
    }
    if (tid == 0) {
        m.start = 0;
        m.after = a.T;
    }
    if (tid < BM / 32) m.bits[tid] = 0;
    __syncthreads();
    // the nearest offsets outside the tile, and those inside as bits
    for (int i = tid; i <= a.sequences; i += blockDim.x) {
        const int at = min(max(a.extents[i], 0), a.T);
        if (at <= row0)
            atomicMax(&m.start, at);
        else if (at < row0 + BM)
            atomicOr(&m.bits[(at - row0) >> 5], 1u << ((at - row0) & 31));
        else
            atomicMin(&m.after, at);
    }
    const int first = min(max(a.extents[0], 0), a.T), behind = min(max(a.extents[a.sequences], 0), a.T);
    real = Span{max(row0, first), min(row0 + BM, behind) - 1};
    __syncthreads();
    if (tid < BM) {
        int start = m.start, end = m.after;
#pragma unroll
        for (int w = 0; w < BM / 32; ++w) {
            const uint32_t at_or_below = w < (tid >> 5) ? ~0u : w == (tid >> 5) ? ~0u >> (31 - (tid & 31)) : 0u;
            const uint32_t below = m.bits[w] & at_or_below;
            if (below) start = row0 + w * 32 + 31 - __clz(below);
        }
#pragma unroll
        for (int w = BM / 32 - 1; w >= 0; --w) {
            const uint32_t above = w > (tid >> 5) ? ~0u : w == (tid >> 5) ? ~(~0u >> (31 - (tid & 31))) : 0u;
            const uint32_t later = m.bits[w] & above;
            if (later) end = row0 + w * 32 + __ffs(later) - 1;
        }
        m.of[tid] = row >= first && row < behind ? Span{start, end - 1} : Span{kNone, kNone};
    }
    __syncthreads();
    return real;
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
    static __device__ __forceinline__ unsigned turned_base() {
        const int lane = threadIdx.x & 63, g = lane >> 4, q = lane & 15;
        const int row = 4 * (g >> 1) + (q >> 2), chunk = (g & 1) * 2 + ((q & 3) >> 1);
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
    // The 4 elements of a row that values 4 i .. 4 i + 3 of a lane of Y^T's tile t are sums of.
    static __device__ __forceinline__ u32x2 four(unsigned tile, int row, int t, int i) {
        const int c = 4 * t + i;
        const unsigned at = tile + row * BYTES + (c / G * G + ((c % G) ^ swizzle(row))) * 16 + ((threadIdx.x & 63) >> 5) * 8;
        return *(const __attribute__((address_space(3))) u32x2*)(size_t)at;
    }
};

// The same address in SGPRs.
__device__ __forceinline__ const char* uniform(const char* p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<const char*>(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) << 32) |
                                         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a));
}

// Direct-to-LDS loads of a tile of BN rows of one tensor, by NW waves. A lane's 16 bytes of
// instruction i land in LDS chunk (wave N + i) 64 + lane, so the source chunk is the one that
// belongs there.
template <int D, int BN, int NW, bool PADDED>
struct TileLoads {
    using R = Rows<D>;
    static constexpr int N = BN * R::CPR / 64 / NW;
    static_assert(N * 64 * NW == BN * R::CPR, "whole instructions");
    uint32_t offset[N];
    __device__ __forceinline__ int row_of(int i) const {
        return (((int)threadIdx.x >> 6) * N + i) * 64 / R::CPR + (((((int)threadIdx.x >> 6) * N + i) * 64) % R::CPR + ((int)threadIdx.x & 63)) / R::CPR;
    }
    __device__ __forceinline__ int chunk_of(int i) const {
        const int at = (((int)threadIdx.x >> 6) * N + i) * 64 + ((int)threadIdx.x & 63);
        const int row = at / R::CPR, slot = at % R::CPR;
        return slot / R::G * R::G + ((slot % R::G) ^ R::swizzle(row));
    }
    __device__ __forceinline__ void init(uint32_t stride) {
#pragma unroll
        for (int i = 0; i < N; ++i) offset[i] = (uint32_t)row_of(i) * stride + (uint32_t)chunk_of(i) * 16;
    }
    // Rows from `from` on (wave-uniform) to LDS address `tile`; rows at or past `count` repeat the last one there is.
    __device__ __forceinline__ void issue(const char* from, uint32_t stride, unsigned tile, int count, int hd) const {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const char* src = uniform(from);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t at = count >= BN ? offset[i] : (uint32_t)min(row_of(i), count - 1) * stride + (uint32_t)chunk_of(i) * 16;
            const unsigned dst = tile + (unsigned)(wave * N + i) * 1024;
            // The wait states: a VMEM instruction that reads an SGPR which VALU wrote needs 5, a
            // direct-to-LDS load after a write of M0 1. Inline, so that the compiler does not wait
            // for the loads of the next tile before it reads this one.
            if (!PADDED || chunk_of(i) * 8 < hd)
                asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(at), "s"(src), "{m0}"(dst) : "memory");
        }
    }
};
// All outstanding loads of this wave have landed.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

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

// The rows of a lane's 16 values of a 32 x 32 product.
__device__ __forceinline__ int value_row(int i) { return (i & 3) + 8 * (i >> 2) + 4 * ((threadIdx.x & 63) >> 5); }

// Values 8 s .. 8 s + 7 of X as operand B of Y^T.
__device__ __forceinline__ bf16x8 as_operand(const f32x16& x, int s) {
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)x[8 * s + i];
    return o;
}

__device__ __forceinline__ bool not_finite(uint32_t bf16) { return (bf16 & 0x7F80u) == 0x7F80u; }
__device__ __forceinline__ bf16x8 only_finite(bf16x8 x) {
    u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (not_finite(w[i])) w[i] &= 0xFFFF0000u;
        if (not_finite(w[i] >> 16)) w[i] &= 0x0000FFFFu;
    }
    return __builtin_bit_cast(bf16x8, w);
}

// X = A B^T for NB blocks of 32 rows of the tile whose plain base is given. Operands are read two
// steps ahead of their products, in groups that the compiler keeps apart: it would read them all at
// once else, into registers that there are not.
template <int D, int NB>
__device__ __forceinline__ void product(f32x16 (&x)[NB], const bf16x8 (&b)[D / 16], unsigned base) {
    using R = Rows<D>;
    constexpr int K = D / 16;
    bf16x8 a[2][2][NB];
    const auto read = [&](int k) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int u = 0; u < NB; ++u) a[(k >> 1) & 1][j][u] = R::plain(base, u, k + j);
    };
#pragma unroll
    for (int u = 0; u < NB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[u][i] = 0.0f;
    read(0);
#pragma unroll
    for (int k = 0; k < K; k += 2) {
        if (k + 2 < K) read(k + 2);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int u = 0; u < NB; ++u)
                x[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[(k >> 1) & 1][j][u], b[k + j], x[u], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Y^T += A'^T X for the tile of 32 NB rows at `tile`, its turned base given.
// Where the mask hides some of the tile's rows from some of the wave's (`edge`), their values in X
// are 0, but 0 times an infinity or NaN is NaN: a product of the tile with zeros tells whether it
// holds any. Then they are left out, and added one by one to the rows that see them.
template <int D, int NB, typename Sees>
__device__ __forceinline__ void add_turned(f32x16 (&y)[D / 32], const f32x16 (&x)[NB], unsigned base, unsigned tile, bool edge,
                                           Sees sees) {
    using R = Rows<D>;
    constexpr int T = D / 32, S = 2 * NB;
    bf16x8 a[2][T];
    const auto read = [&](int s) {
#pragma unroll
        for (int t = 0; t < T; ++t) a[s & 1][t] = R::turned(base, t, s);
    };
    bool all_finite = true;
    if (edge) {
        f32x4 probe = {0, 0, 0, 0};
        const bf16x8 zeros = {};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            read(s);
#pragma unroll
            for (int t = 0; t < T; ++t) probe = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[s & 1][t], zeros, probe, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // a NaN in a row of A makes the product's whole row NaN: each lane has 4 of its rows
        all_finite = !__any(probe[0] != 0.0f || probe[1] != 0.0f || probe[2] != 0.0f || probe[3] != 0.0f);
    }
    if (all_finite) {
        read(0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s + 1 < S) read(s + 1);
            const bf16x8 b = as_operand(x[s >> 1], s & 1);
#pragma unroll
            for (int t = 0; t < T; ++t) y[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[s & 1][t], b, y[t], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bf16x8 b = as_operand(x[s >> 1], s & 1);
#pragma unroll
            for (int t = 0; t < T; ++t) {
                y[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(only_finite(R::turned(base, t, s)), b, y[t], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        for (int row = 0; row < 32 * NB; ++row) {
            const bool see = sees(row);
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x2 e = R::four(tile, row, t, i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t bits = k & 1 ? e[k >> 1] & 0xFFFF0000u : e[k >> 1] << 16;
                        if (see && not_finite(bits >> 16)) y[t][4 * i + k] += __uint_as_float(bits);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
    }
}

// Y^T times `by` (and the lane's row of it) as bf16 to row `to`, elements below hd: a lane and the one
// 32 further exchange halves, so that each stores 16 bytes.
template <int D>
__device__ __forceinline__ void store_turned(__bf16* to, bool there, const f32x16 (&y)[D / 32], float by, int hd) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
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
            const int d = 32 * t + 16 * p + 8 * h;
            if (there && d < hd) *reinterpret_cast<u32x4*>(to + d) = out;
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
__device__ __forceinline__ bool sees(Span s, int at) { return at >= s.first && at <= s.last && s.first != kNone; }

}  // namespace dev
}  // namespace fp
