// Attention over whole prompts (gfx950): the forward pass, and the C ABI
// (include/prompt_attention.h; tiles and operand layouts: prompt_attention.h beside this file).
//
// A wave takes 32 tokens of a query head and passes over the keys that any of its workgroup's
// tokens sees. X = K Q^T, so a lane has half of a tile's logits of one token; the running maximum
// moves only when a logit passes it by 2^8 (probabilities in bf16 keep their relative precision),
// so that between moves lanes exchange nothing. Masks are taken only in tiles where some token
// of the wave does not see some key.
//
// A workgroup is 4 waves of different tokens and tiles of 64 keys, two workgroups a CU, so that one wave's
// products overlap the other's softmax; with few workgroups 2 rows of 4 waves that share the
// tokens and take 32 keys of 128 each (few_workgroups has both sides' times); above heads of 128 the
// registers hold one wave a SIMD and tiles of 32. Short sequences have workgroups without idle waves (short_rows). k and v come by direct-to-LDS loads, two tiles each.
//
// Measured: 8192 tokens, 32 heads on 8 of 128, causal, 549 to 585 us on different cards (power): 940 to 1000 TFLOP/s, 0.8 of a large
// library product's rate. Bound by both units of a SIMD: matrix units busy 4/10 of the time, vector
// units half. At a step that took 575 us it was 504 without the softmax's operations, 408 without the second product, and 473 instead of 598
// on zeros (another card; the clock: power). Heads of 64 have half the products a logit: 2 x 4096 tokens, 5 heads, all see all, 77 us,
// vector units busy half of the time and matrix units a fifth, and 1.25 rounds of workgroups, so that a CU has none for a quarter of it.
#include <cmath>
#include <cstring>
#include <new>

#include "prompt_attention.h"

namespace {

using namespace fp::dev;
using fp::AttentionArgs;

constexpr float kLowest = -3.0e38f;   // the running maximum before any key
constexpr float kSlack = 8.0f;        // how far (log2) a logit may pass it before it moves

__device__ __forceinline__ Place place_of(const AttentionArgs& a) {
    Place p;
    const uint32_t at = in_xcd_order(blockIdx.x, a.blocks);
    const uint32_t rest = fp::fastdiv_u31(at, a.div_group), unit = fp::fastdiv_u31(rest, a.div_tiles);
    p.tile = a.tiles - 1 - (int)(rest - unit * (uint32_t)a.tiles);   // causal: the longest first
    p.batch = (int)fp::fastdiv_u31(unit, a.div_kvh);
    p.kvh = (int)unit - p.batch * a.KVH;
    p.head = p.kvh * a.group + (int)(at - rest * (uint32_t)a.group);
    return p;
}

// Shapes of a workgroup: RW rows of waves with 32 tokens each, and H waves a row that share them and take
// 32 NB keys in turn of each tile of 32 NB H; what they have is joined at the end.
template <int D, bool PADDED, int RW, int H, int NB>
__global__ __launch_bounds__(64 * RW * H, RW * H <= 4 && D <= 128 ? 2 : 1) void attention_kernel(AttentionArgs a) {
    using R = Rows<D>;
    constexpr int NW = RW * H, BM = 32 * RW, BW = 32 * NB, BN = BW * H, TILE = BN * R::BYTES;
    __shared__ __attribute__((aligned(1024))) unsigned char tiles[4 * TILE];   // k, k, v, v
    const int tid = threadIdx.x, lane = tid & 63, place = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = place % RW, turn = H > 1 ? place / RW : 0;
    __shared__ float maxima[H > 1 ? H : 1][BM], sums[H > 1 ? H : 1][BM];
    const unsigned lds = (unsigned)(size_t)(lds_void*)tiles;
    const Place at = place_of(a);
    const int row0 = at.tile * BM, row = row0 + wave * 32 + (lane & 31);

    bf16x8 q[D / 16];
    load_rows<D>(q, a.q + at.batch * a.q_sb + at.head * a.q_sh + (int64_t)min(row, a.T - 1) * a.q_st, row < a.T, a.hd);
    if constexpr (PADDED) {   // the chunks behind hd are never loaded
        for (int i = tid; i < 4 * TILE / 16; i += NW * 64) reinterpret_cast<u32x4*>(tiles)[i] = u32x4{0, 0, 0, 0};
    }
    const Spans spans = find_spans<BM>(a, at.batch, row0, row0 + wave * 32, true, !a.causal);
    Span mine = spans.mine;
    int low = 0, high = -1;
    if (spans.from <= spans.to) {
        low = spans.first.first;
        high = a.causal ? spans.to : spans.last.last;
    }
    const bool there = mine.first != kNone;
    if (a.causal && there) mine.last = row;
    const WaveSight sight = wave_sight(mine);

    f32x16 o[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] = 0.0f;
    float m = kLowest, l = 0.0f;

    const char* k = a.k + at.batch * a.k_sb + at.kvh * a.k_sh;
    const char* v = a.v + at.batch * a.v_sb + at.kvh * a.v_sh;
    TileLoads<D, BN, NW, PADDED> k_loads, v_loads;
    k_loads.init(a.k_st);
    v_loads.init(a.v_st);
    const unsigned plain = R::plain_base(), turned = R::turned_base();
    const auto issue = [&](int p, int set) {
        k_loads.issue(k + (int64_t)p * a.k_st, a.k_st, lds + set * TILE, high + 1 - p, a.hd);
        v_loads.issue(v + (int64_t)p * a.v_st, a.v_st, lds + (2 + set) * TILE, high + 1 - p, a.hd);
    };
    bool left_out = false;
    const auto at_edge = [&](int p) { return p < sight.full_from || p + BW - 1 > sight.full_to; };
    const auto mine_at_edge = [&](int p) { return (p - low) / BW % H == turn && at_edge(p); };
    const auto take = [&](int p, unsigned kt, unsigned vt) {
        const bool edge = at_edge(p);
        f32x16 x[NB];
        product<D, NB, 2>(x, [&](int kk) { return q[kk]; }, kt + plain);
        if (edge) {
            asm volatile("");   // a branch, not selects
#pragma unroll
            for (int u = 0; u < NB; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) x[u][i] = sees(mine, p + 32 * u + value_row(i)) ? x[u][i] : -INFINITY;
        }
        float top = x[0][0];
#pragma unroll
        for (int j = 1; j < 16 * NB; ++j) top = fmaxf(top, x[j >> 4][j & 15]);
        top *= a.scale_log2;
        if (__any(top > m + kSlack)) {
            const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
            const float to = fmaxf(m, fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])));
            const float down = __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= down;
#pragma unroll
            for (int t = 0; t < D / 32; ++t) o[t] *= down;
        }
#pragma unroll
        for (int u = 0; u < NB; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[u][i] = __builtin_amdgcn_exp2f(fmaf(x[u][i], a.scale_log2, -m));
                l += x[u][i];
            }
        bf16x8 w[2 * NB];
        to_operands<NB>(w, x);
        left_out |= add_turned<D, NB, D / 32>(o, w, vt + turned, edge);
    };

    if constexpr (PADDED) {
        wait_lds();
        __syncthreads();
    }
    arrived(q);
    if (low <= high) issue(low, 0);
    int set = 0;
    for (int p = low; p <= high; p += BN, set ^= 1) {
        wait_loads();
        __syncthreads();   // every wave's loads of this tile have landed, and its reads of the other set are done
        if (p + BN <= high) issue(p + BN, set ^ 1);
        const int u = BW * turn;
        if (sight.any && p + u + BW > sight.low && p + u <= sight.high)
            take(p + u, lds + set * TILE + u * R::BYTES, lds + (2 + set) * TILE + u * R::BYTES);
    }

    const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(both[0]) + __uint_as_float(both[1]);
    if constexpr (H > 1) {
        // the row's greatest maximum, and its sum of exponentials
        if (lane < 32) maxima[turn][wave * 32 + lane] = m;
        __syncthreads();
        float to = m;
#pragma unroll
        for (int g = 0; g < H; ++g) to = fmaxf(to, maxima[g][wave * 32 + (lane & 31)]);
        const float down = __builtin_amdgcn_exp2f(m - to);
        m = to;
        if (lane < 32) sums[turn][wave * 32 + lane] = l * down;
#pragma unroll
        for (int t = 0; t < D / 32; ++t) o[t] *= down;
    }
    // behind the last change of the maximum: 0 times an infinity is NaN
    if (left_out) add_left_out<D, BW, false>(o, v, a.v_st, low, high, mine, a.hd, mine_at_edge);
    if constexpr (H > 1) {
        static_assert((H - 1) * RW * 128 * D <= 4 * TILE, "the sums fit the tiles");
        sum_up<D, RW, H>(o, 0, wave, turn, tiles);
        l = 0.0f;
#pragma unroll
        for (int g = 0; g < H; ++g) l += sums[g][wave * 32 + (lane & 31)];
    }
    if (row >= a.T || turn > 0) return;
    if (!there) {
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[t][i] = 0.0f;
    }
    store_turned<D>(a.o + ((int64_t)at.batch * a.T + row) * ((int64_t)a.H * a.hd) + (int64_t)at.head * a.hd, o,
                    there ? 1.0f / l : 0.0f, a.hd);
    if (a.lse && lane < 32)
        a.lse[((int64_t)at.batch * a.H + at.head) * a.T + row] = there ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

template <int D, int RW, int H, int NB>
void launch_shape(const prompt_attention_desc& d, AttentionArgs a, hipStream_t st) {
    a.tiles = (int32_t)((d.tokens + 32 * RW - 1) / (32 * RW));
    a.div_tiles = fp::make_fastdiv_u31((uint32_t)a.tiles);
    a.blocks = (uint32_t)(d.batch * d.n_heads * a.tiles);
    if (d.head_dim == D)
        hipLaunchKernelGGL((attention_kernel<D, false, RW, H, NB>), dim3(a.blocks), dim3(64 * RW * H), 0, st, a);
    else
        hipLaunchKernelGGL((attention_kernel<D, true, RW, H, NB>), dim3(a.blocks), dim3(64 * RW * H), 0, st, a);
}

template <int D>
void launch(const prompt_attention_desc& d, const AttentionArgs& a, hipStream_t st) {
    // workgroups of 128 tokens
    const int64_t blocks = d.batch * d.n_heads * ((d.tokens + 127) / 128);
    const int rows = fp::short_rows(d);
    if (rows == 1)
        launch_shape<D, 1, 1, 1>(d, a, st);
    else if (rows == 2)
        launch_shape<D, 2, 1, 1>(d, a, st);
    else if constexpr (D > 128)
        launch_shape<D, 4, 1, 1>(d, a, st);
    else if (fp::few_workgroups(blocks, d))
        launch_shape<D, 2, 4, 1>(d, a, st);
    else
        launch_shape<D, 4, 1, 2>(d, a, st);
}

}  // namespace

namespace fp {

hipError_t launch_attention(const prompt_attention_desc& d, const AttentionPlan& p, AttentionArgs a, hipStream_t st) {
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

// ---------------------------------------------------------------- C ABI
struct prompt_attention_plan {
    prompt_attention_desc d;
    fp::AttentionPlan p;
    int64_t kvh = 0;
    int device = -1;
};

namespace {

double scale_of(const prompt_attention_desc& d) { return d.sm_scale == 0.0 ? 1.0 / std::sqrt((double)d.head_dim) : d.sm_scale; }

// Elements from a tensor's first to behind its last, or -1 beyond 2^58.
int64_t extent(const int64_t (&s)[3], int64_t b, int64_t heads, int64_t tokens, int64_t hd) {
    const long double n = (long double)(b - 1) * s[0] + (long double)(heads - 1) * s[1] + (long double)(tokens - 1) * s[2] + hd;
    if (n > 0x1p58L) return -1;
    return (b - 1) * s[0] + (heads - 1) * s[1] + (tokens - 1) * s[2] + hd;
}

// What the backward pass keeps of each token and head, in whole pieces of 16 bytes.
size_t stats_bytes(const fp::AttentionPlan& p) { return ((size_t)p.rows * 8 + 15) / 16 * 16; }

int check(const prompt_attention_desc* d, fp::AttentionPlan* out, int64_t* kvh_out) {
    if (!d) return FUSED_PROJ_EINVAL;
    if (d->dtype != FUSED_PROJ_BF16 && d->dtype != FUSED_PROJ_F32) return FUSED_PROJ_EINVAL;
    if (d->causal != 0 && d->causal != 1) return FUSED_PROJ_EINVAL;
    if (d->batch < 0 || d->tokens < 1 || d->n_heads < 1 || d->head_dim < 1 || d->sequences < 0) return FUSED_PROJ_EINVAL;
    if (d->n_kv_heads < 0 || (d->n_kv_heads > 0 && d->n_heads % d->n_kv_heads != 0)) return FUSED_PROJ_EINVAL;
    if (d->sequences > 0 && d->batch != 1) return FUSED_PROJ_EINVAL;
    const double factor = scale_of(*d) * 1.4426950408889634;
    if (!(d->sm_scale >= 0.0) || !(factor < 0x1p128) || !(factor >= 0x1p-126) || std::isinf((float)factor)) return FUSED_PROJ_EINVAL;
    for (const int64_t* s : {d->q_strides, d->k_strides, d->v_strides})
        for (int i = 0; i < 3; ++i)
            if (s[i] < 0) return FUSED_PROJ_EINVAL;
    if (d->dtype != FUSED_PROJ_BF16 || d->head_dim % 8 != 0 || d->head_dim > 256) return FUSED_PROJ_EUNSUPPORTED;
    const int64_t lim = (int64_t(1) << 31) - 1, kvh = d->n_kv_heads > 0 ? d->n_kv_heads : d->n_heads;
    if (d->tokens >= (1 << 30) || d->sequences >= (1 << 30) || d->batch > lim || d->n_heads > lim) return FUSED_PROJ_EUNSUPPORTED;
    if (d->batch * d->n_heads > lim / d->tokens) return FUSED_PROJ_EUNSUPPORTED;
    // a launch has below 2^32 threads, and none more than 512 for 64 tokens of a head
    if (d->batch * d->n_heads >= (int64_t(1) << 23) / ((d->tokens + 63) / 64)) return FUSED_PROJ_EUNSUPPORTED;
    for (const int64_t* s : {d->q_strides, d->k_strides, d->v_strides}) {
        for (int i = 0; i < 3; ++i)
            if (s[i] % 8 != 0) return FUSED_PROJ_EUNSUPPORTED;
        if (s[2] > (1 << 24)) return FUSED_PROJ_EUNSUPPORTED;
    }
    if (d->n_heads * d->head_dim > (1 << 24)) return FUSED_PROJ_EUNSUPPORTED;   // o's token stride
    const int64_t b = d->batch > 0 ? d->batch : 1;
    if (extent(d->q_strides, b, d->n_heads, d->tokens, d->head_dim) < 0 || extent(d->k_strides, b, kvh, d->tokens, d->head_dim) < 0 ||
        extent(d->v_strides, b, kvh, d->tokens, d->head_dim) < 0)
        return FUSED_PROJ_EUNSUPPORTED;
    fp::AttentionPlan p;
    for (const int dim : {32, 64, 96, 128, 192, 256})
        if (d->head_dim <= dim) {
            p.dim = dim;
            break;
        }
    p.rows = d->batch * d->tokens * d->n_heads;
    fp::plan_attention_backward(*d, kvh, &p);
    p.backward_workspace = stats_bytes(p);
    if (p.kv_parts > 1) p.backward_workspace += (size_t)p.kv_parts * 2 * (size_t)(d->batch * kvh * d->tokens * d->head_dim) * 4;
    if (out) *out = p;
    if (kvh_out) *kvh_out = kvh;
    return FUSED_PROJ_OK;
}

struct Range {
    uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes}; }
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

int hip_status(hipError_t e) {
    if (e == hipSuccess) return FUSED_PROJ_OK;
    fp::set_last_hip_error(e);
    return FUSED_PROJ_EHIP;
}

// The checks of a call, and the arguments that both passes share. outs first in `r`.
int prepare(const prompt_attention_plan* h, const void* q, const void* k, const void* v, const int32_t* extents, Range* r,
            int n_out, int n, AttentionArgs* out) {
    const prompt_attention_desc& d = h->d;
    if (!q || !k || !v || (!extents && d.sequences > 0)) return FUSED_PROJ_EINVAL;
    const Range in[4] = {range(q, extent(d.q_strides, d.batch, d.n_heads, d.tokens, d.head_dim) * 2),
                         range(k, extent(d.k_strides, d.batch, h->kvh, d.tokens, d.head_dim) * 2),
                         range(v, extent(d.v_strides, d.batch, h->kvh, d.tokens, d.head_dim) * 2),
                         range(extents, extents ? (d.sequences > 0 ? d.sequences + 1 : d.batch) * 4 : 0)};
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v) & 15u || (uintptr_t)extents & 3u) return FUSED_PROJ_EALIGN;
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n; ++j)
            if (overlap(r[i], r[j])) return FUSED_PROJ_EALIAS;
        for (const Range& x : in)
            if (overlap(r[i], x)) return FUSED_PROJ_EALIAS;
    }
    int dev = -1;
    const int rc = hip_status(hipGetDevice(&dev));
    if (rc) return rc;
    if (dev != h->device) return FUSED_PROJ_EINVAL;
    AttentionArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = static_cast<const char*>(q);
    a.k = static_cast<const char*>(k);
    a.v = static_cast<const char*>(v);
    a.extents = extents;
    a.q_sb = d.q_strides[0] * 2;
    a.q_sh = d.q_strides[1] * 2;
    a.q_st = (uint32_t)(d.q_strides[2] * 2);
    a.k_sb = d.k_strides[0] * 2;
    a.k_sh = d.k_strides[1] * 2;
    a.k_st = (uint32_t)(d.k_strides[2] * 2);
    a.v_sb = d.v_strides[0] * 2;
    a.v_sh = d.v_strides[1] * 2;
    a.v_st = (uint32_t)(d.v_strides[2] * 2);
    a.o_st = (uint32_t)(d.n_heads * d.head_dim * 2);
    a.batch = (int32_t)d.batch;
    a.T = (int32_t)d.tokens;
    a.H = (int32_t)d.n_heads;
    a.KVH = (int32_t)h->kvh;
    a.hd = (int32_t)d.head_dim;
    a.group = a.H / a.KVH;
    a.sequences = (int32_t)d.sequences;
    a.causal = d.causal;
    a.scale = (float)scale_of(d);
    a.scale_log2 = (float)(scale_of(d) * 1.4426950408889634);
    a.div_group = fp::make_fastdiv_u31((uint32_t)a.group);
    a.div_kvh = fp::make_fastdiv_u31((uint32_t)a.KVH);
    *out = a;
    return FUSED_PROJ_OK;
}

}  // namespace

extern "C" {

int prompt_attention_validate(const prompt_attention_desc* desc) { return check(desc, nullptr, nullptr); }

int prompt_attention_create(const prompt_attention_desc* desc, prompt_attention_t* out) {
    if (!out) return FUSED_PROJ_EINVAL;
    *out = nullptr;
    fp::AttentionPlan p;
    int64_t kvh = 0;
    int rc = check(desc, &p, &kvh);
    if (rc) return rc;
    prompt_attention_plan* h = new (std::nothrow) prompt_attention_plan();
    if (!h) return FUSED_PROJ_EHIP;
    h->d = *desc;
    h->p = p;
    h->kvh = kvh;
    rc = hip_status(hipGetDevice(&h->device));
    if (rc) {
        delete h;
        return rc;
    }
    *out = h;
    return FUSED_PROJ_OK;
}

int prompt_attention_backward_workspace_size(prompt_attention_t h, size_t* bytes) {
    if (!h || !bytes) return FUSED_PROJ_EINVAL;
    *bytes = h->p.backward_workspace;
    return FUSED_PROJ_OK;
}

int prompt_attention_run(prompt_attention_t h, const void* q, const void* k, const void* v, const int32_t* extents, void* o,
                         void* lse, void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (h->p.rows == 0) return FUSED_PROJ_OK;
    if (!o) return FUSED_PROJ_EINVAL;
    if ((uintptr_t)o & 15u || (uintptr_t)lse & 3u) return FUSED_PROJ_EALIGN;
    Range r[2] = {range(o, h->p.rows * h->d.head_dim * 2), range(lse, lse ? h->p.rows * 4 : 0)};
    AttentionArgs a;
    const int rc = prepare(h, q, k, v, extents, r, 2, 2, &a);
    if (rc) return rc;
    a.o = static_cast<__bf16*>(o);
    a.lse = static_cast<float*>(lse);
    return hip_status(fp::launch_attention(h->d, h->p, a, static_cast<hipStream_t>(stream)));
}

int prompt_attention_backward(prompt_attention_t h, const void* q, const void* k, const void* v, const int32_t* extents,
                              const void* o, const void* lse, const void* d_o, void* dq, void* dk, void* dv, void* workspace,
                              size_t workspace_bytes, void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    if (h->p.rows == 0) return FUSED_PROJ_OK;
    const size_t need = h->p.backward_workspace;
    if (!o || !lse || !d_o || !dq || !dk || !dv || !workspace || workspace_bytes < need) return FUSED_PROJ_EINVAL;
    if (((uintptr_t)o | (uintptr_t)d_o | (uintptr_t)dq | (uintptr_t)dk | (uintptr_t)dv | (uintptr_t)workspace) & 15u || (uintptr_t)lse & 3u)
        return FUSED_PROJ_EALIGN;
    const int64_t q_bytes = h->p.rows * h->d.head_dim * 2, kv_bytes = h->d.batch * h->kvh * h->d.tokens * h->d.head_dim * 2;
    Range r[7] = {range(dq, q_bytes), range(dk, kv_bytes), range(dv, kv_bytes), range(workspace, (int64_t)need),
                  range(o, q_bytes), range(d_o, q_bytes), range(lse, h->p.rows * 4)};
    AttentionArgs a;
    const int rc = prepare(h, q, k, v, extents, r, 4, 7, &a);
    if (rc) return rc;
    a.o_in = static_cast<const __bf16*>(o);
    a.lse_in = static_cast<const float*>(lse);
    a.d_o = static_cast<const char*>(d_o);
    a.dq = static_cast<__bf16*>(dq);
    a.dk = static_cast<__bf16*>(dk);
    a.dv = static_cast<__bf16*>(dv);
    a.stats = static_cast<float*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats_bytes(h->p));
    return hip_status(fp::launch_attention_backward(h->d, h->p, a, static_cast<hipStream_t>(stream)));
}

int prompt_attention_destroy(prompt_attention_t h) {
    delete h;
    return FUSED_PROJ_OK;
}

}  // extern "C"
