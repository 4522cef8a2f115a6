// The backward pass of attention over whole prompts (gfx950; formulas are in
// include/prompt_attention.h, tiles and operand layouts in prompt_attention.h beside this file).
//
// Two kernels, both with the logits computed again. The first passes over the keys like the
// forward pass, for 128 tokens of a query head, and leaves dq; it also leaves D and lse log2(e) of its
// tokens for the second. The second passes over the tokens that see 128 keys, head after head of
// the group, and leaves dk and dv. 9 products, 4 and 5 (those with ds count twice, as it is two numbers), where 7 would do in one
// kernel: there dq would be summed by atomics, in an order that changes from run to run, or
// through partial sums in memory.
//
// D_i is sum_j p_ij dp_ij. What the caller has of o is rounded to bf16, and ds = p (dp - D) is a difference: with D from that o
// alone dq and dk were off by 0.0040 of their norm at 2 tokens and 0.0030 at 8 (heads of 128, causal, normal inputs), where
// their own rounding is 0.0017. The ds of a row sum to 0 if D is right, so their sum is what D lacks, and the first kernel
// leaves the second a D with that sum added. For dq itself it comes too late; rows that see few keys, where it matters most, get it
// beforehand (kFewKeys).
#include "prompt_attention.h"

namespace {

using namespace fp::dev;
using fp::AttentionArgs;

// Rows that see at most this many keys have their D corrected before dq is formed, by two products more for these keys. In other
// rows what o's rounding leaves in dq falls with the root of the number of keys that their softmax spreads over, but for what these keys
// have in common. 512 tokens, causal, normal inputs: dq is off by 0.0020 of its norm without any of it, by 0.0017 with; logits three times as
// steep, 0.0030 and 0.0025; 32 x 512 ragged, all see all, keys with a common part, 0.0022 and 0.0022; 0.0017 if all rows were corrected. Times,
// us, none / these / all rows: forward and backward of 2 x 4096 tokens, 32 heads on 8 of 128, causal, 1522 / 1526 / 1788, of 32 x 512 ragged,
// 12 of 64, 145 / 145 / 164; backward of 256 x 128, 32 on 8 of 128, causal, 532 / 582 / 582, of 512 x 7, 176 / 191 / 191.
constexpr int kFewKeys = 128;

// Shapes of a workgroup: RW rows of waves with 32 tokens each, and H waves a row that share them and take S
// times 32 keys in turn of each tile of 32 H S; their sums are added at the end.
template <int D, bool PADDED, int RW, int H, int S>
__global__ __launch_bounds__(64 * RW * H, RW * H <= 4 && D <= 128 ? 2 : 1) void attention_dq_kernel(AttentionArgs a) {
    using R = Rows<D>;
    constexpr int NW = RW * H, BM = 32 * RW, BN = 32 * H * S, TILE = BN * R::BYTES;
    __shared__ __attribute__((aligned(1024))) unsigned char tiles[4 * TILE];   // k, k, v, v
    const int tid = threadIdx.x, lane = tid & 63, place = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = place % RW, turn = H > 1 ? place / RW : 0;
    const unsigned lds = (unsigned)(size_t)(lds_void*)tiles;
    const uint32_t order = in_xcd_order(blockIdx.x, a.blocks);
    const uint32_t rest = fp::fastdiv_u31(order, a.div_group), unit = fp::fastdiv_u31(rest, a.div_tiles);
    const int batch = (int)fp::fastdiv_u31(unit, a.div_kvh), kvh = (int)unit - batch * a.KVH;
    const int head = kvh * a.group + (int)(order - rest * (uint32_t)a.group);
    const int row0 = (a.tiles - 1 - (int)(rest - unit * (uint32_t)a.tiles)) * BM;   // causal: the longest first
    const int row = row0 + wave * 32 + (lane & 31), row_in = min(row, a.T - 1);

    bf16x8 q[D / 16], d_o[D / 16];
    const char* do_row = a.d_o + ((int64_t)batch * a.T + row_in) * a.o_st + (int64_t)head * a.hd * 2;
    load_rows<D>(q, a.q + batch * a.q_sb + head * a.q_sh + (int64_t)row_in * a.q_st, row < a.T, a.hd);
    load_rows<D>(d_o, do_row, row < a.T, a.hd);
    const int64_t stat = ((int64_t)batch * a.H + head) * a.T + row_in;
    float lse = a.lse_in[stat] * kLog2e, delta = 0.0f;
    {
        const char* o_row = reinterpret_cast<const char*>(a.o_in) + (do_row - a.d_o);
        bf16x8 o[D / 16];
        load_rows<D>(o, o_row, row < a.T, a.hd);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 8; ++i) delta = fmaf((float)o[kk][i], (float)d_o[kk][i], delta);
        const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(delta), __float_as_uint(delta), false, false);
        delta = __uint_as_float(both[0]) + __uint_as_float(both[1]);
    }
    if constexpr (PADDED) {   // the chunks behind hd are never loaded
        for (int i = tid; i < 4 * TILE / 16; i += NW * 64) reinterpret_cast<u32x4*>(tiles)[i] = u32x4{0, 0, 0, 0};
    }
    const Spans spans = find_spans<BM>(a, batch, row0, row0 + wave * 32, true, !a.causal);
    Span mine = spans.mine;
    int low = 0, high = -1;
    if (spans.from <= spans.to) {
        low = spans.first.first;
        high = a.causal ? spans.to : spans.last.last;
    }
    const bool there = mine.first != kNone;
    if (a.causal && there) mine.last = row;
    const WaveSight sight = wave_sight(mine);
    if (!there) lse = delta = 0.0f;
    const bool is_few = there && mine.last - mine.first < kFewKeys;
    const Span few = is_few ? mine : Span{kNone, kNone};
    const WaveSight few_sight = wave_sight(few);
    const Span few_keys = of_workgroup<NW>(few_sight.any ? Span{few_sight.low, few_sight.high} : Span{kNone, -1});

    f32x16 dq[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[t][i] = 0.0f;

    const char* k = a.k + batch * a.k_sb + kvh * a.k_sh;
    const char* v = a.v + batch * a.v_sb + kvh * a.v_sh;
    TileLoads<D, BN, NW, PADDED> k_loads, v_loads;
    k_loads.init(a.k_st);
    v_loads.init(a.v_st);
    const unsigned plain = R::plain_base(), turned = R::turned_base();
    const auto issue = [&](int p, int set, int last) __attribute__((always_inline)) {
        k_loads.issue(k + (int64_t)p * a.k_st, a.k_st, lds + set * TILE, last + 1 - p, a.hd);
        v_loads.issue(v + (int64_t)p * a.v_st, a.v_st, lds + (2 + set) * TILE, last + 1 - p, a.hd);
    };
    float missing = 0.0f;   // what D lacks: the sum of this lane's ds
    const auto ds_of = [&](f32x16 (&x)[1], int p, unsigned kt, unsigned vt, Span span, bool edge) __attribute__((always_inline)) {
        f32x16 y[1];
        product<D, 1, 2>(x, [&](int kk) { return q[kk]; }, kt + plain);
        product<D, 1, 2>(y, [&](int kk) { return d_o[kk]; }, vt + plain);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[0][i] = __builtin_amdgcn_exp2f(fmaf(x[0][i], a.scale_log2, -lse)) * (y[0][i] - delta);
        if (edge) {
            asm volatile("");   // a branch, not selects
#pragma unroll
            for (int i = 0; i < 16; ++i) x[0][i] = sees(span, p + value_row(i)) ? x[0][i] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) missing += x[0][i];
    };
    // `missing` of both halves of a row and of its H waves, in one order. Between two calls lies a barrier of the loop over the tiles.
    __shared__ float parts[H > 1 ? H : 1][BM];
    const auto add_missing = [&](bool to_mine) __attribute__((always_inline)) {
        const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(missing), __float_as_uint(missing), false, false);
        float sum = __uint_as_float(both[0]) + __uint_as_float(both[1]);
        if constexpr (H > 1) {
            if (lane < 32) parts[turn][wave * 32 + lane] = sum;
            __syncthreads();
            sum = 0.0f;
#pragma unroll
            for (int g = 0; g < H; ++g) sum += parts[g][wave * 32 + (lane & 31)];
        }
        if (to_mine) delta += sum;
        missing = 0.0f;
    };
    bool left_out = false;
    const auto at_edge = [&](int p) { return p < sight.full_from || p + 31 > sight.full_to; };
    const auto mine_at_edge = [&](int p) { return (p - low) / 32 % H == turn && at_edge(p); };
    const auto take = [&](int p, unsigned kt, unsigned vt) __attribute__((always_inline)) {
        const bool edge = at_edge(p);
        f32x16 x[1];
        ds_of(x, p, kt, vt, mine, edge);
        bf16x8 w[2];
        to_operands<1>(w, x);
        bf16x8 rest[2];
        rest_to_operands<1>(rest, w, x);
        left_out |= add_turned<D, 1, D / 32>(dq, w, kt + turned, edge, rest);
    };

    if constexpr (PADDED) {
        wait_lds();
        __syncthreads();
    }
    arrived(q);
    arrived(d_o);
    asm volatile("" : "+v"(lse), "+v"(delta));
    // The tiles from `from` to `last`, by the waves whose rows see some of them.
    const auto over_tiles = [&](int from, int last, const WaveSight& s, auto f) __attribute__((always_inline)) {
        int set = 0;
        for (int p = from; p <= last; p += BN, set ^= 1) {
            wait_loads();
            __syncthreads();   // every wave's loads of this tile have landed, and its reads of the other set are done
            if (p + BN <= last) issue(p + BN, set ^ 1, last);
            for (int u = 32 * turn; u < BN; u += 32 * H)
                if (s.any && p + u + 32 > s.low && p + u <= s.high)
                    f(p + u, lds + set * TILE + u * R::BYTES, lds + (2 + set) * TILE + u * R::BYTES);
        }
    };
    bool loaded = false;
    if (few_keys.first <= few_keys.last) {
        issue(few_keys.first, 0, few_keys.last);
        over_tiles(few_keys.first, few_keys.last, few_sight, [&](int p, unsigned kt, unsigned vt) __attribute__((always_inline)) {
            f32x16 x[1];
            ds_of(x, p, kt, vt, few, p < few_sight.full_from || p + 31 > few_sight.full_to);
        });
        add_missing(is_few);
        wait_loads();
        __syncthreads();   // the tiles are read
        loaded = few_keys.first == low && few_keys.last == high && high - low < BN;   // the only tile is there already
    }
    if (low <= high && !loaded) issue(low, 0, high);
    over_tiles(low, high, sight, take);
    add_missing(there);
    if (row < a.T && lane < 32 && turn == 0) {
        a.stats[stat] = lse;
        a.stats[(int64_t)a.H * a.T * a.batch + stat] = delta;
    }

    // a logit of -infinity has a ds of 0, and 0 times an infinity is NaN
    if (left_out) add_left_out<D, 32, true>(dq, k, a.k_st, low, high, mine, a.hd, mine_at_edge);
    if constexpr (H > 1) {
        static_assert((H - 1) * RW * 128 * D <= 4 * TILE, "the sums fit the tiles");
        sum_up<D, RW, H>(dq, 0, wave, turn, tiles);
    }
    if (row >= a.T || turn > 0) return;
    if (!there) {
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) dq[t][i] = 0.0f;
    }
    store_turned<D>(a.dq + (((int64_t)batch * a.H + head) * a.T + row) * a.hd, dq, a.scale, a.hd);
}

// Shapes of a workgroup: RW rows of waves with 32 keys each, and H waves a row that share these keys and
// take S times 32 tokens in turn of each tile of 32 H S; their sums are added at the end. Heads above 128: two
// waves have the same keys and tokens, and every other 32 elements of dk and dv (PARTS); both
// compute P and ds. One wave with all of them has no registers for a second on its SIMD, and at 256 not for itself.
template <int D, bool PADDED, int RW, int H, int S, int PARTS>
__global__ __launch_bounds__(64 * RW * H * PARTS, RW * H * PARTS <= 4 && D <= 96 ? 2 : 1) void attention_dkv_kernel(AttentionArgs a) {
    using R = Rows<D>;
    // Heads of 128 and more: the accumulators, k and v leave no registers for two waves a SIMD (heads above 128: for one), so v's rows
    // stay in LDS.
    constexpr bool V_IN_LDS = D >= 128;
    constexpr int NW = RW * H * PARTS, BM = 32 * RW, BN = 32 * H * S, TILE = BN * R::BYTES, T = D / 32 / PARTS;
    __shared__ __attribute__((aligned(1024))) unsigned char tiles[4 * TILE + (V_IN_LDS ? BM * R::BYTES : 0)];   // q, q, do, do, v
    __shared__ __attribute__((aligned(16))) float stats[2][2][BN];             // set; lse log2(e), D; token
    const int tid = threadIdx.x, lane = tid & 63, place = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = place % RW, turn = H > 1 ? place / RW % H : 0, part = PARTS > 1 ? place / (RW * H) : 0;
    const unsigned lds = (unsigned)(size_t)(lds_void*)tiles;
    const uint32_t order = in_xcd_order(blockIdx.x, a.blocks);
    const uint32_t unit = fp::fastdiv_u31(order, a.div_tiles);
    const int batch = (int)fp::fastdiv_u31(unit, a.div_kvh), kvh = (int)unit - batch * a.KVH;
    const int row0 = (int)(order - unit * (uint32_t)a.tiles) * BM;   // causal: the first keys are seen by most
    const int row = row0 + wave * 32 + (lane & 31), row_in = min(row, a.T - 1);

    const int first_head = (int)blockIdx.y * a.part_heads, behind_head = min(first_head + a.part_heads, a.group);   // of the group

    bf16x8 k[D / 16], v[V_IN_LDS ? 1 : D / 16];
    load_rows<D>(k, a.k + batch * a.k_sb + kvh * a.k_sh + (int64_t)row_in * a.k_st, row < a.T, a.hd);
    const char* v_head = a.v + batch * a.v_sb + kvh * a.v_sh;
    if constexpr (!V_IN_LDS) load_rows<D>(v, v_head + (int64_t)row_in * a.v_st, row < a.T, a.hd);
    if constexpr (PADDED) {   // the chunks behind hd are never loaded
        for (int i = tid; i < (int)sizeof(tiles) / 16; i += NW * 64) reinterpret_cast<u32x4*>(tiles)[i] = u32x4{0, 0, 0, 0};
    }
    const Spans spans = find_spans<BM>(a, batch, row0, row0 + wave * 32, !a.causal, true);
    Span mine = spans.mine;   // the tokens that see this lane's key
    int low = 0, high = -1;
    if (spans.from <= spans.to) {
        low = a.causal ? spans.from : spans.first.first;
        high = spans.last.last;
    }
    const bool there = mine.first != kNone;
    if (a.causal && there) mine.first = row;
    const WaveSight sight = wave_sight(mine);

    f32x16 dk[T], dv[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[t][i] = dv[t][i] = 0.0f;

    TileLoads<D, BN, NW, PADDED, D < 128> q_loads, do_loads;
    q_loads.init(a.q_st);
    do_loads.init(a.o_st);
    const unsigned plain = R::plain_base(), turned = R::turned_base(part);
    const auto issue = [&](int g, int p, int set) {
        const int head = kvh * a.group + g, count = high + 1 - p;
        q_loads.issue(a.q + batch * a.q_sb + head * a.q_sh + (int64_t)p * a.q_st, a.q_st, lds + set * TILE, count, a.hd);
        do_loads.issue(a.d_o + ((int64_t)batch * a.T + p) * a.o_st + (int64_t)head * a.hd * 2, a.o_st, lds + (2 + set) * TILE, count, a.hd);
        // a number a lane: BN of lse, then BN of D
        static_assert(2 * BN % 64 == 0 && 2 * BN <= 64 * NW, "whole waves");
        if (place * 64 < 2 * BN) {
            int at = threadIdx.x;
            asm volatile("" : "+v"(at));   // what follows from it is not kept since the last tile
            const float* from = a.stats + (at < BN ? 0 : (int64_t)a.H * a.T * a.batch) + ((int64_t)batch * a.H + head) * a.T + p +
                                min(at & (BN - 1), count - 1);
            const unsigned dst = (unsigned)(size_t)(lds_void*)&stats[set][0][0] + (unsigned)place * 256;
            asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, off" ::"v"(from), "{m0}"(dst) : "memory");
        }
    };
    bool left_out = false;
    const auto at_edge = [&](int p) { return p < sight.full_from || p + 31 > sight.full_to; };
    const auto mine_at_edge = [&](int p) { return (p - low) / 32 % H == turn && at_edge(p); };
    const auto take = [&](int p, unsigned qt, unsigned dt, const float* lse, const float* delta) {
        const bool edge = at_edge(p);
        f32x16 x[1], y[1];
        constexpr int C = T == 4 && D >= 128 ? 2 : T, J = D >= 128 ? 1 : 2;
        bf16x8 w[2], dw[2], rest[2];
        {
            const int h = lane >> 5;
            product<D, 1, J>(
                y, [&](int kk) { return V_IN_LDS ? R::plain(lds + 4 * TILE + wave * 32 * R::BYTES + plain, 0, kk) : v[V_IN_LDS ? 0 : kk]; },
                dt + plain);
            product<D, 1, J>(x, [&](int kk) { return k[kk]; }, qt + plain);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 l = *reinterpret_cast<const f32x4*>(lse + 8 * j + 4 * h);
                const f32x4 d = *reinterpret_cast<const f32x4*>(delta + 8 * j + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[0][4 * j + i] = __builtin_amdgcn_exp2f(fmaf(x[0][4 * j + i], a.scale_log2, -l[i]));
                    y[0][4 * j + i] = x[0][4 * j + i] * (y[0][4 * j + i] - d[i]);
                }
            }
            if (edge) {
                asm volatile("");   // a branch, not selects
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool see = sees(mine, p + value_row(i));
                    x[0][i] = see ? x[0][i] : 0.0f;
                    y[0][i] = see ? y[0][i] : 0.0f;
                }
            }
            to_operands<1>(w, x);
            to_operands<1>(dw, y);
            rest_to_operands<1>(rest, dw, y);
            __builtin_amdgcn_sched_barrier(0);
        }
        left_out |= add_turned<D, 1, C, PARTS>(dv, w, dt + turned, edge);
        // where a token's q is not finite neither is its lse, so that ds is NaN for every key that it sees
        add_turned<D, 1, C, PARTS>(dk, dw, qt + turned, edge, rest);
    };

    if constexpr (PADDED) {
        wait_lds();
        __syncthreads();
    }
    arrived(k);
    if constexpr (!V_IN_LDS) arrived(v);
    int set = 0;
    if (low <= high) {
        if constexpr (V_IN_LDS) {   // rows behind the last token repeat it
            TileLoads<D, BM, NW, PADDED, false> v_loads;
            v_loads.init(a.v_st);
            v_loads.issue(v_head + (int64_t)row0 * a.v_st, a.v_st, lds + 4 * TILE, min(BM, a.T - row0), a.hd);
        }
        issue(first_head, low, 0);
        int g = first_head, p = low;
        while (g < behind_head) {
            int next_g = g, next_p = p + BN;
            if (next_p > high) {
                next_p = low;
                ++next_g;
            }
            wait_loads();
            __syncthreads();   // every wave's loads of this tile have landed, and its reads of the other set are done
            if (next_g < behind_head) issue(next_g, next_p, set ^ 1);
            for (int u = 32 * turn; u < BN; u += 32 * H)
                if (sight.any && p + u + 32 > sight.low && p + u <= sight.high)
                    take(p + u, lds + set * TILE + u * R::BYTES, lds + (2 + set) * TILE + u * R::BYTES, &stats[set][0][u], &stats[set][1][u]);
            set ^= 1;
            g = next_g;
            p = next_p;
        }
    }

    if (left_out)
        for (int g = first_head; g < behind_head; ++g)
            add_left_out<D, 32, false, PARTS>(dv, a.d_o + (int64_t)batch * a.T * a.o_st + (int64_t)(kvh * a.group + g) * a.hd * 2, a.o_st, low, high,
                                       mine, a.hd, mine_at_edge, part);
    if constexpr (H > 1) {
        static_assert((H - 1) * RW * 128 * D <= 4 * TILE, "the sums fit the tiles");
        sum_up<D / PARTS, RW * PARTS, H>(dk, 0, part * RW + wave, turn, tiles);
        sum_up<D / PARTS, RW * PARTS, H>(dv, 1, part * RW + wave, turn, tiles);
    }
    if (row >= a.T) return;
    const int64_t to = (((int64_t)batch * a.KVH + kvh) * a.T + row) * a.hd;
    const auto store = [&](__bf16* out, f32x16 (&y)[T], float by) {
        if (!there) {
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) y[t][i] = 0.0f;
        }
        if (a.partial) {
            float* const sums = a.partial + ((int64_t)blockIdx.y * 2 + (out == a.dv)) * ((int64_t)a.batch * a.KVH * a.T * a.hd) + to;
#pragma unroll
            for (int i = 0; i < 4 * T; ++i) {
                const int d = 32 * ((i >> 2) * PARTS + part) + 8 * (i & 3) + 4 * (lane >> 5);
                if (d < a.hd)
                    *reinterpret_cast<f32x4*>(sums + d) = f32x4{y[i >> 2][4 * (i & 3)], y[i >> 2][4 * (i & 3) + 1], y[i >> 2][4 * (i & 3) + 2], y[i >> 2][4 * (i & 3) + 3]};
            }
        } else {
            store_turned<D, PARTS>(out + to, y, by, a.hd, part);
        }
    };
    if (H == 1 || turn == 0) store(a.dk, dk, a.scale);
    if (H == 1 || turn == 1) store(a.dv, dv, 1.0f);
}

// Workgroups of 128 keys are few for longer than those of tokens: a group's heads are in one, and with a causal mask the first
// has twice the mean's work. dq and dk, dv, heads of 64, us, with 4 rows of one wave / 4 of 2 / 2 of 4 (dq as it is best):
//   4 x 512 tokens, 12 heads (192 workgroups)  47 / 45 / 49         8 x 512, 12 heads (384)  59 / 67 / 67     16 x 512 (768)  90 / 101 / 111
//   16 x 2048 (256)     135 / 117 / 119          causal             106 / 92 / 75
//   32 x 2048 (512)     193 / 200 / 210          causal             161 / 164 / 146       16 x 4096, causal (512)  282 / 233 / 238
// and heads of 128, which have registers for one wave a SIMD of 4 rows of one, causal:
//   16 x 2048 (256)     163 / 134 / 116          16 x 4096 (512)    459 / 409 / 425       32 x 2048 (512)  303 / 256 / 235
int64_t few_key_blocks(const prompt_attention_desc& d) { return d.tokens < 1024 ? 160 : d.causal ? 512 : 256; }

// Adds up the parts of dk and dv, 4 elements a thread.
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, int parts, int64_t n) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const int dv = blockIdx.y;
    const float* from = a.partial + dv * n + i;
    f32x4 sum = *reinterpret_cast<const f32x4*>(from);
    for (int p = 1; p < parts; ++p) sum += *reinterpret_cast<const f32x4*>(from + (int64_t)p * 2 * n);
    const float by = dv ? 1.0f : a.scale;
    bf16x4 o;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = (__bf16)(sum[k] * by);
    *reinterpret_cast<bf16x4*>((dv ? a.dv : a.dk) + i) = o;
}

template <int D, int RW, int H, int S, int PARTS = 1>
void launch_dkv(const prompt_attention_desc& d, const fp::AttentionPlan& p, AttentionArgs a, hipStream_t st) {
    a.tiles = (int32_t)((d.tokens + 32 * RW - 1) / (32 * RW));
    a.div_tiles = fp::make_fastdiv_u31((uint32_t)a.tiles);
    a.blocks = (uint32_t)(d.batch * a.KVH * a.tiles);
    const dim3 grid(a.blocks, (unsigned)p.kv_parts);
    if (d.head_dim == D)
        hipLaunchKernelGGL((attention_dkv_kernel<D, false, RW, H, S, PARTS>), grid, dim3(64 * RW * H * PARTS), 0, st, a);
    else
        hipLaunchKernelGGL((attention_dkv_kernel<D, true, RW, H, S, PARTS>), grid, dim3(64 * RW * H * PARTS), 0, st, a);
}

template <int D, int RW, int H, int S>
void launch_dq(const prompt_attention_desc& d, AttentionArgs a, hipStream_t st) {
    a.tiles = (int32_t)((d.tokens + 32 * RW - 1) / (32 * RW));
    a.div_tiles = fp::make_fastdiv_u31((uint32_t)a.tiles);
    a.blocks = (uint32_t)(d.batch * d.n_heads * a.tiles);
    if (d.head_dim == D)
        hipLaunchKernelGGL((attention_dq_kernel<D, false, RW, H, S>), dim3(a.blocks), dim3(64 * RW * H), 0, st, a);
    else
        hipLaunchKernelGGL((attention_dq_kernel<D, true, RW, H, S>), dim3(a.blocks), dim3(64 * RW * H), 0, st, a);
}

template <int D>
void launch(const prompt_attention_desc& d, const fp::AttentionPlan& p, AttentionArgs a, hipStream_t st) {
    const int rows = fp::short_rows(d);
    if (rows == 1) {
        launch_dq<D, 1, 1, 1>(d, a, st);
        launch_dkv<D, 1, 1, 1, D <= 128 ? 1 : 2>(d, p, a, st);
        return;
    }
    if (rows == 2) {
        launch_dq<D, 2, 1, 1>(d, a, st);
        launch_dkv<D, 2, 1, 1, D <= 128 ? 1 : 2>(d, p, a, st);
        return;
    }
    // workgroups of 128 tokens
    const int64_t blocks = d.batch * d.n_heads * ((d.tokens + 127) / 128);
    if constexpr (D > 128)
        launch_dq<D, 4, 1, 1>(d, a, st);
    else if (fp::few_workgroups(blocks, d))
        launch_dq<D, 2, 4, 1>(d, a, st);
    else
        launch_dq<D, 4, 1, 2>(d, a, st);
    const int64_t kv_blocks = blocks / a.group, few = few_key_blocks(d);
    if constexpr (D == 256)
        launch_dkv<D, 2, 1, 1, 2>(d, p, a, st);
    else if constexpr (D == 192)
        launch_dkv<D, 2, 2, 1, 2>(d, p, a, st);
    else if (kv_blocks < few)
        launch_dkv<D, 2, 4, 1>(d, p, a, st);
    else if (D == 128 || kv_blocks < 2 * few)
        launch_dkv<D, 4, 2, 1>(d, p, a, st);
    else
        launch_dkv<D <= 96 ? D : 96, 4, 1, 2>(d, p, a, st);
}

}  // namespace

namespace fp {

void plan_attention_backward(const prompt_attention_desc& d, int64_t kvh, AttentionPlan* p) {
    // Where the workgroups are of 64 keys and still fewer than twice the CUs (one is on a CU at a time), a group's heads are cut into parts;
    // their sums go through memory. The whole backward pass, causal, without and with parts: 32 heads on 8 of 128, 512 tokens 67 and 47 us,
    // 2048 tokens 253 and 209; 16 on 4 of 256, 1024 tokens 389 and 168. Parts are of whole heads, the number of a part rounded up, so there may be
    // fewer workgroups than wanted (2999 tokens, 16 heads on 4: 376).
    const int64_t group = d.n_heads / kvh, blocks = d.batch * kvh * ((d.tokens + 63) / 64);
    const bool small = p->dim > 128 || d.batch * kvh * ((d.tokens + 127) / 128) < few_key_blocks(d);
    p->kv_parts = 1;
    if (small && blocks > 0 && blocks < 512 && d.tokens >= 256) {
        const int64_t wanted = (512 + blocks - 1) / blocks, heads = (group + wanted - 1) / wanted;
        p->kv_parts = (int32_t)((group + heads - 1) / heads);
    }
}

hipError_t launch_attention_backward(const prompt_attention_desc& d, const AttentionPlan& p, AttentionArgs a, hipStream_t st) {
    a.part_heads = (a.group + p.kv_parts - 1) / p.kv_parts;
    if (p.kv_parts == 1) a.partial = nullptr;
    switch (p.dim) {
        case 32: launch<32>(d, p, a, st); break;
        case 64: launch<64>(d, p, a, st); break;
        case 96: launch<96>(d, p, a, st); break;
        case 128: launch<128>(d, p, a, st); break;
        case 192: launch<192>(d, p, a, st); break;
        default: launch<256>(d, p, a, st);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.kv_parts == 1) return e;
    const int64_t n = d.batch * a.KVH * d.tokens * d.head_dim;
    hipLaunchKernelGGL(attention_join_kernel, dim3((unsigned)((n / 4 + 255) / 256), 2), dim3(256), 0, st, a, p.kv_parts, n);
    return hipGetLastError();
}

}  // namespace fp
