// The backward pass of attention over whole prompts (gfx950; formulas are in
// include/prompt_attention.h, tiles and operand layouts in prompt_attention.h beside this file).
//
// Two kernels, both with the logits computed again. The first passes over the keys like the
// forward pass, for 128 tokens of a query head, and leaves dq; it also leaves D and lse log2(e) of its
// tokens for the second. The second passes over the tokens that see 128 keys, head after head of
// the group, and leaves dk and dv. 7 products of the forward pass's size where 5 would do in one
// kernel: there dq would be summed by atomics, in an order that changes from run to run, or
// through partial sums in memory.
#include "prompt_attention.h"

namespace {

using namespace fp::dev;
using fp::AttentionArgs;

constexpr int kWaves = 4, kRows = 32 * kWaves;
constexpr int64_t kFewBlocks = 192, kManyBlocks = 512;

template <int D, bool PADDED>
__global__ __launch_bounds__(kWaves * 64, D <= 128 ? 2 : 1) void attention_dq_kernel(AttentionArgs a) {
    using R = Rows<D>;
    constexpr int BN = D <= 128 ? 64 : 32, TILE = BN * R::BYTES;
    __shared__ __attribute__((aligned(1024))) unsigned char tiles[4 * TILE];   // k, k, v, v
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const unsigned lds = (unsigned)(size_t)(lds_void*)tiles;
    const uint32_t order = in_xcd_order(blockIdx.x, a.blocks);
    const uint32_t rest = fp::fastdiv_u31(order, a.div_group), unit = fp::fastdiv_u31(rest, a.div_tiles);
    const int batch = (int)fp::fastdiv_u31(unit, a.div_kvh), kvh = (int)unit - batch * a.KVH;
    const int head = kvh * a.group + (int)(order - rest * (uint32_t)a.group);
    const int row0 = (a.tiles - 1 - (int)(rest - unit * (uint32_t)a.tiles)) * kRows;   // causal: the longest first
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
        for (int i = tid; i < 4 * TILE / 16; i += kWaves * 64) reinterpret_cast<u32x4*>(tiles)[i] = u32x4{0, 0, 0, 0};
    }
    const Spans spans = find_spans<kRows>(a, batch, row0, row0 + wave * 32);
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
    if (row < a.T && lane < 32) {
        a.stats[stat] = lse;
        a.stats[(int64_t)a.H * a.T * a.batch + stat] = delta;
    }

    f32x16 dq[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[t][i] = 0.0f;

    const char* k = a.k + batch * a.k_sb + kvh * a.k_sh;
    const char* v = a.v + batch * a.v_sb + kvh * a.v_sh;
    TileLoads<D, BN, kWaves, PADDED> k_loads, v_loads;
    k_loads.init(a.k_st);
    v_loads.init(a.v_st);
    const unsigned plain = R::plain_base(), turned = R::turned_base();
    const auto issue = [&](int p, int set) {
        k_loads.issue(k + (int64_t)p * a.k_st, a.k_st, lds + set * TILE, high + 1 - p, a.hd);
        v_loads.issue(v + (int64_t)p * a.v_st, a.v_st, lds + (2 + set) * TILE, high + 1 - p, a.hd);
    };
    bool left_out = false;
    const auto at_edge = [&](int p) { return p < sight.full_from || p + 31 > sight.full_to; };
    const auto take = [&](int p, unsigned kt, unsigned vt) {
        const bool edge = at_edge(p);
        f32x16 x[1], y[1];
        product<D, 1, 2>(x, [&](int kk) { return q[kk]; }, kt + plain);
        product<D, 1, 2>(y, [&](int kk) { return d_o[kk]; }, vt + plain);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[0][i] = __builtin_amdgcn_exp2f(fmaf(x[0][i], a.scale_log2, -lse)) * (y[0][i] - delta);
        if (edge) {
            asm volatile("");   // a branch, not selects
#pragma unroll
            for (int i = 0; i < 16; ++i) x[0][i] = sees(mine, p + value_row(i)) ? x[0][i] : 0.0f;
        }
        bf16x8 w[2];
        to_operands<1>(w, x);
        left_out |= add_turned<D, 1, D / 32>(dq, w, kt + turned, edge);
    };

    if constexpr (PADDED) __syncthreads();
    arrived(q);
    arrived(d_o);
    asm volatile("" : "+v"(lse), "+v"(delta));
    if (low <= high) issue(low, 0);
    int set = 0;
    for (int p = low; p <= high; p += BN, set ^= 1) {
        wait_loads();
        __syncthreads();   // every wave's loads of this tile have landed, and its reads of the other set are done
        if (p + BN <= high) issue(p + BN, set ^ 1);
        for (int u = 0; u < BN; u += 32)
            if (sight.any && p + u + 32 > sight.low && p + u <= sight.high)
                take(p + u, lds + set * TILE + u * R::BYTES, lds + (2 + set) * TILE + u * R::BYTES);
    }

    // a logit of -infinity has a ds of 0, and 0 times an infinity is NaN
    if (left_out) add_left_out<D, 32, true>(dq, k, a.k_st, low, high, mine, a.hd, at_edge);
    if (row >= a.T) return;
    if (!there) {
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) dq[t][i] = 0.0f;
    }
    store_turned<D>(a.dq + (((int64_t)batch * a.H + head) * a.T + row) * a.hd, true, dq, a.scale, a.hd);
}

// Shapes of a workgroup: R rows of waves with 32 keys each, and H waves a row that share these keys and
// take 32 tokens in turn of each tile of 32 H; their sums are added at the end.
template <int D, bool PADDED, int RW, int H>
__global__ __launch_bounds__(64 * RW * H, 1) void attention_dkv_kernel(AttentionArgs a) {
    using R = Rows<D>;
    // Heads of 128 and more: the accumulators, k and v leave no registers for two waves a SIMD (heads above 128: for one), so v's rows
    // stay in LDS.
    constexpr bool V_IN_LDS = D >= 128;
    constexpr int NW = RW * H, BM = 32 * RW, BN = 32 * H, TILE = BN * R::BYTES;
    __shared__ __attribute__((aligned(1024))) unsigned char tiles[4 * TILE + (V_IN_LDS ? BM * R::BYTES : 0)];   // q, q, do, do, v
    __shared__ __attribute__((aligned(16))) float stats[2][2][BN];             // set; lse log2(e), D; token
    const int tid = threadIdx.x, lane = tid & 63, place = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = place % RW, turn = place / RW;
    const unsigned lds = (unsigned)(size_t)(lds_void*)tiles;
    const uint32_t order = in_xcd_order(blockIdx.x, a.blocks);
    const uint32_t unit = fp::fastdiv_u31(order, a.div_tiles);
    const int batch = (int)fp::fastdiv_u31(unit, a.div_kvh), kvh = (int)unit - batch * a.KVH;
    const int row0 = (int)(order - unit * (uint32_t)a.tiles) * BM;   // causal: the first keys are seen by most
    const int row = row0 + wave * 32 + (lane & 31), row_in = min(row, a.T - 1);

    bf16x8 k[D / 16], v[V_IN_LDS ? 1 : D / 16];
    load_rows<D>(k, a.k + batch * a.k_sb + kvh * a.k_sh + (int64_t)row_in * a.k_st, row < a.T, a.hd);
    const char* v_head = a.v + batch * a.v_sb + kvh * a.v_sh;
    if constexpr (!V_IN_LDS) load_rows<D>(v, v_head + (int64_t)row_in * a.v_st, row < a.T, a.hd);
    if constexpr (PADDED) {   // the chunks behind hd are never loaded
        for (int i = tid; i < (int)sizeof(tiles) / 16; i += NW * 64) reinterpret_cast<u32x4*>(tiles)[i] = u32x4{0, 0, 0, 0};
    }
    const Spans spans = find_spans<BM>(a, batch, row0, row0 + wave * 32);
    Span mine = spans.mine;   // the tokens that see this lane's key
    int low = 0, high = -1;
    if (spans.from <= spans.to) {
        low = a.causal ? spans.from : spans.first.first;
        high = spans.last.last;
    }
    const bool there = mine.first != kNone;
    if (a.causal && there) mine.first = row;
    const WaveSight sight = wave_sight(mine);

    f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[t][i] = dv[t][i] = 0.0f;

    TileLoads<D, BN, NW, PADDED, D < 128> q_loads, do_loads;
    q_loads.init(a.q_st);
    do_loads.init(a.o_st);
    const unsigned plain = R::plain_base(), turned = R::turned_base();
    // threads 0 .. BN - 1 fetch lse, BN .. 2 BN - 1 fetch D of the next tile
    const auto issue = [&](int g, int p, int set) -> float {
        const int head = kvh * a.group + g, count = high + 1 - p;
        float s = 0.0f;
        if (tid < 2 * BN) {
            const int64_t at = ((int64_t)batch * a.H + head) * a.T + p + min(tid & (BN - 1), count - 1);
            s = a.stats[(tid < BN ? 0 : (int64_t)a.H * a.T * a.batch) + at];
        }
        q_loads.issue(a.q + batch * a.q_sb + head * a.q_sh + (int64_t)p * a.q_st, a.q_st, lds + set * TILE, count, a.hd);
        do_loads.issue(a.d_o + ((int64_t)batch * a.T + p) * a.o_st + (int64_t)head * a.hd * 2, a.o_st, lds + (2 + set) * TILE, count, a.hd);
        return s;
    };
    const auto keep = [&](int set, float s) {
        if (tid < 2 * BN) stats[set][tid / BN][tid & (BN - 1)] = s;
    };
    bool left_out = false;
    const auto at_edge = [&](int p) { return p < sight.full_from || p + 31 > sight.full_to; };
    const auto mine_at_edge = [&](int p) { return (p - low) / 32 % H == turn && at_edge(p); };
    const auto take = [&](int p, unsigned qt, unsigned dt, const float* lse, const float* delta) {
        const bool edge = at_edge(p);
        f32x16 x[1], y[1];
        constexpr int C = D / 32 % 2 == 0 && D >= 128 ? 2 : D / 32, J = D >= 128 ? 1 : 2;
        bf16x8 w[2], dw[2];
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
            __builtin_amdgcn_sched_barrier(0);
        }
        left_out |= add_turned<D, 1, C>(dv, w, dt + turned, edge);
        // where a token's q is not finite neither is its lse, so that ds is NaN for every key that it sees
        add_turned<D, 1, C>(dk, dw, qt + turned, edge);
    };

    if constexpr (PADDED) __syncthreads();
    arrived(k);
    if constexpr (!V_IN_LDS) arrived(v);
    int set = 0;
    if (low <= high) {
        if constexpr (V_IN_LDS) {   // rows behind the last token repeat it
            TileLoads<D, BM, NW, PADDED, false> v_loads;
            v_loads.init(a.v_st);
            v_loads.issue(v_head + (int64_t)row0 * a.v_st, a.v_st, lds + 4 * TILE, min(BM, a.T - row0), a.hd);
        }
        const float s = issue(0, low, 0);
        keep(0, s);
        int g = 0, p = low;
        while (g < a.group) {
            int next_g = g, next_p = p + BN;
            if (next_p > high) {
                next_p = low;
                ++next_g;
            }
            wait_loads();
            __syncthreads();   // every wave's loads of this tile have landed, and its reads of the other set are done
            float next = 0.0f;
            if (next_g < a.group) next = issue(next_g, next_p, set ^ 1);
            const int u = 32 * turn;
            if (sight.any && p + u + 32 > sight.low && p + u <= sight.high)
                take(p + u, lds + set * TILE + u * R::BYTES, lds + (2 + set) * TILE + u * R::BYTES, &stats[set][0][u], &stats[set][1][u]);
            keep(set ^ 1, next);
            set ^= 1;
            g = next_g;
            p = next_p;
        }
    }

    if (left_out)
        for (int g = 0; g < a.group; ++g)
            add_left_out<D, 32, false>(dv, a.d_o + (int64_t)batch * a.T * a.o_st + (int64_t)(kvh * a.group + g) * a.hd * 2, a.o_st, low, high,
                                       mine, a.hd, mine_at_edge);
    if constexpr (H > 1) {
        // a row's sums: its first wave takes dk, its second dv, from what the others leave in the tiles' place
        f32x4* const shared = reinterpret_cast<f32x4*>(tiles) + wave * D * 8 + lane;
        constexpr int NEXT = RW * D * 8;   // the next wave of the row
        const auto sum_up = [&](f32x16 (&y)[D / 32], int taker) {
            __syncthreads();   // the tiles, or the last sums, are read
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
        };
        static_assert((H - 1) * NEXT * 16 <= 4 * TILE, "the sums fit the tiles");
        sum_up(dk, 0);
        sum_up(dv, 1);
    }
    if (row >= a.T) return;
    const int64_t to = (((int64_t)batch * a.KVH + kvh) * a.T + row) * a.hd;
    const auto store = [&](__bf16* out, f32x16 (&y)[D / 32], float by) {
        if (!there) {
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) y[t][i] = 0.0f;
        }
        store_turned<D>(out + to, true, y, by, a.hd);
    };
    if (H == 1 || turn == 0) store(a.dk, dk, a.scale);
    if (H == 1 || turn == 1) store(a.dv, dv, 1.0f);
}

template <int D, int RW, int H>
void launch_dkv(const prompt_attention_desc& d, AttentionArgs a, hipStream_t st) {
    a.tiles = (int32_t)((d.tokens + 32 * RW - 1) / (32 * RW));
    a.div_tiles = fp::make_fastdiv_u31((uint32_t)a.tiles);
    a.blocks = (uint32_t)(d.batch * a.KVH * a.tiles);
    if (d.head_dim == D)
        hipLaunchKernelGGL((attention_dkv_kernel<D, false, RW, H>), dim3(a.blocks), dim3(64 * RW * H), 0, st, a);
    else
        hipLaunchKernelGGL((attention_dkv_kernel<D, true, RW, H>), dim3(a.blocks), dim3(64 * RW * H), 0, st, a);
}

template <int D>
void launch(const prompt_attention_desc& d, AttentionArgs a, hipStream_t st) {
    a.tiles = (int32_t)((d.tokens + kRows - 1) / kRows);
    a.div_tiles = fp::make_fastdiv_u31((uint32_t)a.tiles);
    a.blocks = (uint32_t)(d.batch * d.n_heads * a.tiles);
    if (d.head_dim == D)
        hipLaunchKernelGGL((attention_dq_kernel<D, false>), dim3(a.blocks), dim3(kWaves * 64), 0, st, a);
    else
        hipLaunchKernelGGL((attention_dq_kernel<D, true>), dim3(a.blocks), dim3(kWaves * 64), 0, st, a);
    // workgroups of 128 keys
    const int64_t blocks = d.batch * a.KVH * ((d.tokens + 127) / 128);
    if constexpr (D > 128)
        launch_dkv<D, 4, 1>(d, a, st);
    else if (blocks < kFewBlocks)
        launch_dkv<D, 2, 4>(d, a, st);
    else if (D == 128 || blocks < kManyBlocks)
        launch_dkv<D, 4, 2>(d, a, st);
    else
        launch_dkv<D <= 96 ? D : 96, 4, 1>(d, a, st);
}

}  // namespace

namespace fp {

hipError_t launch_attention_backward(const prompt_attention_desc& d, const AttentionPlan& p, AttentionArgs a, hipStream_t st) {
    switch (p.dim) {
        case 32: launch<32>(d, a, st); break;
        case 64: launch<64>(d, a, st); break;
        case 96: launch<96>(d, a, st); break;
        case 128: launch<128>(d, a, st); break;
        case 192: launch<192>(d, a, st); break;
        default: launch<256>(d, a, st);
    }
    return hipGetLastError();
}

}  // namespace fp
