// Layer norm over the channels of a channels-first or token-major activation, forward and
// backward (gfx950; the formulas are in layer_norm.h).
//
// The op moves bytes: forward reads x and writes y, backward reads x and dy and writes dx,
// with about 10 and 20 VALU operations a value where the memory rate allows 28 and 42. Each
// tensor is touched once, where a row or strip fits a workgroup's registers: a token's channels
// stay there (as stored, unpacked again for each use) between the sums over them and the output
// that needs the sums. Channels-first, more than 1536 channels or slabs shorter than a strip do
// not, and are read again for each use.
//
// Token-major rows: TPR threads (a wave, or a workgroup of 256 or 1024) hold a row, NCH
// 16-byte pieces each. Channels-first: a workgroup holds a strip of TL * V tokens with all
// channels; TL neighbouring lanes read TL * 16 contiguous bytes of one channel.
//
// The variance is the mean square of x - mean, from the held values: no cancellation.
// dgamma and dbeta: every thread keeps its channels' sums in fp32 over the rows or strips
// that its workgroup takes in turn; the workgroup's sums go to the workspace and a second
// kernel adds them in 64 bits, in a fixed order.
//
// Measured (a large copy reaches 5.2 TB/s): forward 24 x 768 x 1024 bf16 channels-first 16.6 us
// (4.6 TB/s), 3063 rows of 1387 fp32 8.6 us (4.0 TB/s); backward 16384 rows of 768 bf16 16 us
// (4.7 TB/s), 24 x 1408 x 1024 bf16 channels-first 57 us (3.6 TB/s); column sums 3 to 5 us. Rows
// that leave a wave mostly idle, 131072 of 24 bf16: 33 us (0.4 TB/s), backward 41; strips that
// are read again, 24 x 2048 x 1024 bf16: 69 us (2.9 TB/s), backward 113.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <type_traits>

#include "../../include/layer_norm.h"
#include "fused_proj_kernels.h"
#include "vector_io.h"

namespace {

using namespace fp::dev;

struct NormArgs {
    const void* x;
    const void* gamma;
    const void* beta;      // nullptr without a bias
    const void* dy;        // backward
    void* y;               // y, or dx
    float* mean;           // [b*S]; forward: nullptr when not wanted
    float* rstd;
    float* partial;        // backward: [workgroups, 2, C]
    int64_t x_sb, x_ss, x_sc;   // element strides of x
    int32_t M, S, C;
    int32_t strips;        // channels-first: strips of a slab
    int32_t all_strips;    // and of all of them
    float inv_c, eps;
    fp::FastDivU31 div_s;  // token -> slab; channels-first: strip -> slab (by strips)
};

// ------------------------------------------------------------------ token-major rows
// Sum over the TPR threads of a row, the same bits in each; `red` holds a value a wave.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) v += red[w];
        __syncthreads();
    }
    return v;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const NormArgs& a, int row) {
    const int bi = (int)fp::fastdiv_u31((uint32_t)row, a.div_s);
    return static_cast<const T*>(a.x) + (int64_t)bi * a.x_sb + (int64_t)(row - bi * a.S) * a.x_ss;
}

template <typename T, int NCH, int TPR, bool TAIL>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void layer_norm_rows_kernel(NormArgs a) {
    constexpr int V = Piece<T>::V, BLOCK = TPR < 256 ? 256 : TPR, RPB = BLOCK / TPR;
    __shared__ float red[TPR > 64 ? TPR / 64 : 1];
    const int lane = threadIdx.x % TPR;
    // only the last piece can end past the row (NCH is the least that covers it, but at 1024)
    const auto whole = [](int i) { return !TAIL || (TPR < 1024 && i < NCH - 1); };
    const T* gamma = static_cast<const T*>(a.gamma);
    const T* beta = static_cast<const T*>(a.beta);
    for (int row = blockIdx.x * RPB + threadIdx.x / TPR; row < a.M; row += gridDim.x * RPB) {
        const T* x = row_of<T>(a, row);
        u32x4 h[NCH];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * TPR + lane) * V;
            h[i] = u32x4{0, 0, 0, 0};
            if ((TPR < 1024 && i < NCH - 1) || c < a.C) h[i] = load_piece(x + c, a.C - c, whole(i));
        }
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) sum += Piece<T>::get(h[i], e);   // past C: zeros
        const float mean = row_sum<TPR>(sum, red) * a.inv_c;
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int n = a.C - (i * TPR + lane) * V;
            unpack_again(h[i]);
            if (n > 0) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = Piece<T>::get(h[i], e) - mean;
                    if (whole(i) || e < n) sq = fmaf(d, d, sq);
                }
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(sq, red) * a.inv_c + a.eps);
        T* y = static_cast<T*>(a.y) + (int64_t)row * a.C;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * TPR + lane) * V, n = a.C - c;
            unpack_again(h[i]);
            if (n > 0) {
                const u32x4 g = load_piece(gamma + c, n, whole(i));
                const u32x4 b = beta ? load_piece(beta + c, n, whole(i)) : u32x4{0, 0, 0, 0};
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o[e] = fmaf((Piece<T>::get(h[i], e) - mean) * rstd, Piece<T>::get(g, e), Piece<T>::get(b, e));
                store_piece<T>(y + c, o, n, whole(i));
            }
        }
        if (a.mean && lane == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

// As for the strips below, the registers of a row's pieces take the next row's as its dx is
// written, and nothing else is loaded in between.
template <typename T, int NCH, int TPR, bool TAIL>
__global__ __launch_bounds__(TPR < 512 ? 512 : TPR) void layer_norm_rows_grad_kernel(NormArgs a) {
    constexpr int V = Piece<T>::V, BLOCK = TPR < 512 ? 512 : TPR, RPB = BLOCK / TPR, WPR = TPR / 64;
    __shared__ float red[BLOCK / 64 * 2];
    __shared__ float both[RPB > 1 ? 2 * NCH * TPR * V : 1];
    constexpr bool kAhead = TPR < 1024;   // a workgroup of 1024 has too few registers for it
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const auto whole = [](int i) { return !TAIL || (TPR < 1024 && i < NCH - 1); };
    const auto left = [&](int i) { return a.C - (i * TPR + lane) * V; };   // values of the row from the piece on
    const auto inside = [&](int i) { return (TPR < 1024 && i < NCH - 1) || left(i) > 0; };
    u32x4 hx[NCH], hd[NCH], hg[NCH];
    float dg[NCH][V], db[NCH][V];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        hg[i] = inside(i) ? load_piece(static_cast<const T*>(a.gamma) + (i * TPR + lane) * V, left(i), whole(i)) : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < V; ++e) dg[i][e] = db[i][e] = 0.0f;
    }
    const T* x;
    const T* dy;
    float mean_next = 0.0f, rstd_next = 0.0f;
    const auto go_to = [&](int row) {
        x = row_of<T>(a, row);
        dy = static_cast<const T*>(a.dy) + (int64_t)row * a.C;
        mean_next = a.mean[row];
        rstd_next = a.rstd[row];
    };
    const auto load = [&](int i) {
        hx[i] = load_piece(x + (i * TPR + lane) * V, left(i), whole(i));
        hd[i] = load_piece(dy + (i * TPR + lane) * V, left(i), whole(i));
    };
    const int row0 = blockIdx.x * RPB + sub, turn = gridDim.x * RPB;
    if (row0 < a.M) go_to(row0);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        hx[i] = hd[i] = u32x4{0, 0, 0, 0};
        if (row0 < a.M && inside(i)) load(i);
    }
    // every row slot of the workgroup takes the same number of turns, so that its barriers meet
    for (int row = row0; row - sub < a.M; row += turn) {
        const bool real = row < a.M;
        const float mean = mean_next, rstd = rstd_next;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            if (real && inside(i)) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (whole(i) || e < left(i)) {
                        const float d = Piece<T>::get(hd[i], e), xh = (Piece<T>::get(hx[i], e) - mean) * rstd;
                        const float gd = d * Piece<T>::get(hg[i], e);
                        s1 += gd;
                        s2 = fmaf(gd, xh, s2);
                        dg[i][e] = fmaf(d, xh, dg[i][e]);
                        db[i][e] += d;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                settle(dg[i][e]);
                settle(db[i][e]);
            }
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if constexpr (TPR > 64) {
            const int wave = threadIdx.x >> 6, row_wave = wave / WPR * WPR;
            if ((threadIdx.x & 63) == 0) {
                red[2 * wave] = s1;
                red[2 * wave + 1] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) {
                s1 += red[2 * (row_wave + w)];
                s2 += red[2 * (row_wave + w) + 1];
            }
            __syncthreads();
        }
        // dx = rstd (d gamma - c1 - xhat c2) = d gamma rstd + (x - mean) t2 + t1
        const float t1 = -rstd * (s1 * a.inv_c), t2 = -rstd * (rstd * (s2 * a.inv_c));
        T* dx = static_cast<T*>(a.y) + (int64_t)row * a.C;
        const bool more = row + turn < a.M;
        if (more) go_to(row + turn);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            unpack_again(hx[i]);
            unpack_again(hd[i]);
            if (real && inside(i)) {
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o[e] = fmaf(Piece<T>::get(hx[i], e) - mean, t2, fmaf(Piece<T>::get(hd[i], e) * Piece<T>::get(hg[i], e), rstd, t1));
                store_piece<T>(dx + (i * TPR + lane) * V, o, left(i), whole(i));
                if (kAhead && more) load(i);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!kAhead && more) {
#pragma unroll
            for (int i = 0; i < NCH; ++i)
                if (inside(i)) load(i);
        }
    }
    // the workgroup's sums: its row slots add theirs in turn
    float* out = a.partial + (int64_t)blockIdx.x * 2 * a.C;
    if constexpr (RPB > 1) {
        for (int r = 0; r < RPB; ++r) {
            if (sub == r) {
#pragma unroll
                for (int i = 0; i < NCH; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int at = (i * TPR + lane) * V + e;
                        both[at] = r == 0 ? dg[i][e] : both[at] + dg[i][e];
                        both[NCH * TPR * V + at] = r == 0 ? db[i][e] : both[NCH * TPR * V + at] + db[i][e];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.C; c += BLOCK) {
            out[c] = both[c];
            out[a.C + c] = both[NCH * TPR * V + c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int c = (i * TPR + lane) * V + e;
                if (c < a.C) {
                    out[c] = dg[i][e];
                    out[a.C + c] = db[i][e];
                }
            }
    }
}

// ------------------------------------------------------------------ channels-first strips
constexpr int TL = 4;   // lanes along the tokens: 64 bytes of a channel

// A workgroup's strip is TL * V tokens of one slab. Thread (cr, tl) holds V tokens of the
// channels cr, cr + R, cr + 2R, ... (R = threads / TL).
//
// Sum of f[e] over the lanes of a wave with the same tl (lane bits 2..5): each exchange halves the values a lane carries, so the sums of 8 values cost 4 + 2 + 1
// exchanges instead of 24. The lane's remaining value is the sum for token `lane_token`.
template <int V>
__device__ __forceinline__ float strip_sum(const float (&f)[V]) {
    float r;
    if constexpr (V == 8) {
        const float a0 = swap_sum32(f[0], f[4]), a1 = swap_sum32(f[1], f[5]);
        const float a2 = swap_sum32(f[2], f[6]), a3 = swap_sum32(f[3], f[7]);
        const float b0 = swap_sum16(a0, a2), b1 = swap_sum16(a1, a3);
        const bool odd = threadIdx.x & 8;
        r = (odd ? b1 : b0) + dpp<kRowRor8>(odd ? b0 : b1);
    } else {
        const float a0 = swap_sum32(f[0], f[2]), a1 = swap_sum32(f[1], f[3]);
        r = swap_sum16(a0, a1);
        r += dpp<kRowRor8>(r);
    }
    r += dpp<0x1B>(dpp<kHalfMirror>(r));   // lane ^ 7, then ^ 3: lane ^ 4
    return r;
}
template <int V>
__device__ __forceinline__ int lane_token() {
    const int l = threadIdx.x & 63, b5 = l >> 5, b4 = (l >> 4) & 1, b3 = (l >> 3) & 1;
    return (l & (TL - 1)) * V + (V == 8 ? b5 * 4 + b4 * 2 + b3 : b5 * 2 + b4);
}

// Sums of NS sets of per-token values over the whole workgroup: tot[set][token], the same
// bits for every thread. `red`: [waves][NS][TL * V].
template <int V, int NS, int NT>
__device__ __forceinline__ void strip_total(const float (&f)[NS][V], float* red, float* tot) {
    constexpr int TT = TL * V, W = NT / 64;
    const int t = lane_token<V>();
#pragma unroll
    for (int s = 0; s < NS; ++s) red[((threadIdx.x >> 6) * NS + s) * TT + t] = strip_sum<V>(f[s]);
    __syncthreads();
    if (threadIdx.x < NS * TT) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += red[w * NS * TT + threadIdx.x];
        tot[threadIdx.x] = v;
    }
    __syncthreads();
}

// Workgroups are dispatched round-robin over the 8 XCDs, each with its own L2. Strips that
// share cache lines (neighbours in a slab) go to workgroups of one XCD.
__device__ __forceinline__ int strip_of(int bid, int grid) {
    const int xcd = bid & 7, q = grid >> 3, r = grid & 7;
    return xcd * q + min(xcd, r) + (bid >> 3);
}

// The strips of a slab cover its tokens from the first on; the last one is moved back to end
// with the slab, so that every piece is whole. Its first tokens are then the strip before's
// too: both compute and store the same bits, and dgamma and dbeta count them once. EDGE: the
// slab is shorter than a strip, and pieces end with it.
template <int TT, bool EDGE>
__device__ __forceinline__ void strip_tokens(const NormArgs& a, int strip, int& bi, int& first, int& twice) {
    bi = (int)fp::fastdiv_u31((uint32_t)strip, a.div_s);
    first = (strip - bi * a.strips) * TT;
    twice = 0;
    if (!EDGE && first + TT > a.S) {
        twice = first + TT - a.S;
        first = a.S - TT;
    }
}

// The thread's piece of channel i R + cr: bytes from the slab, a base that the whole workgroup
// shares; 32 bits of them where the strip is held (the plan has checked that the slab fits),
// so that no 64-bit address a piece takes registers.
template <int NCH>
using Offset = std::conditional_t<(NCH > 0), uint32_t, uint64_t>;
template <typename T, typename O>
__device__ __forceinline__ T* at_bytes(T* base, O off) {
    return reinterpret_cast<T*>(reinterpret_cast<char*>(const_cast<std::remove_const_t<T>*>(base)) + off);
}

// NCH > 0: the strip is held in registers, NCH pieces a thread (all but the last within C).
// NCH = 0 (more channels than that, or EDGE): it is read again for each use, from the caches.
template <typename T, int NCH, int NT, bool EDGE>
__global__ __launch_bounds__(NT) void layer_norm_strips_kernel(NormArgs a) {
    static_assert(!EDGE || NCH == 0, "pieces that end with the slab are not held");
    constexpr int V = Piece<T>::V, R = NT / TL, TT = TL * V, HOLD = NCH > 0 ? NCH : 1;
    __shared__ float red[NT / 64 * TT];
    __shared__ float tot[2][TT];
    const int tl = threadIdx.x % TL, cr = threadIdx.x / TL;
    const uint32_t bid = blockIdx.y * gridDim.x + blockIdx.x;   // rows of kMostBlocks
    if (bid >= (uint32_t)a.all_strips) return;
    int bi, first, twice;
    strip_tokens<TT, EDGE>(a, strip_of((int)bid, a.all_strips), bi, first, twice);
    const int n = EDGE ? a.S - first - tl * V : V;
    const int nch = NCH > 0 ? NCH : (a.C + R - 1) / R;
    const T* x = static_cast<const T*>(a.x) + (int64_t)bi * a.x_sb + first;
    T* y = static_cast<T*>(a.y) + (int64_t)bi * a.C * a.S + first;
    const auto off_x = [&](int i) { return ((Offset<NCH>)(i * R + cr) * (Offset<NCH>)a.x_sc + tl * V) * (Offset<NCH>)sizeof(T); };
    const auto off_y = [&](int i) { return ((Offset<NCH>)(i * R + cr) * (Offset<NCH>)a.S + tl * V) * (Offset<NCH>)sizeof(T); };
    const auto inside = [&](int i) { return ((NCH > 0 && i < NCH - 1) || i * R + cr < a.C) && (!EDGE || n > 0); };
    u32x4 h[HOLD];
    const auto load = [&](int i) {
        return inside(i) ? load_piece(at_bytes(x, off_x(i)), n, !EDGE) : u32x4{0, 0, 0, 0};
    };
    if constexpr (NCH > 0) {
#pragma unroll
        for (int i = 0; i < HOLD; ++i) h[i] = load(i);
    }
    const auto piece = [&](int i) {
        if constexpr (NCH > 0) {
            unpack_again(h[i]);
            return h[i];
        } else {
            return load(i);
        }
    };
    float f[1][V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[0][e] = 0.0f;
#pragma unroll NCH > 0 ? NCH : 1
    for (int i = 0; i < nch; ++i) {
        const u32x4 p = piece(i);
#pragma unroll
        for (int e = 0; e < V; ++e) f[0][e] += Piece<T>::get(p, e);
    }
    strip_total<V, 1, NT>(f, red, tot[0]);
    float mean[V], rstd[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        mean[e] = tot[0][tl * V + e] * a.inv_c;
        f[0][e] = 0.0f;
    }
#pragma unroll NCH > 0 ? NCH : 1
    for (int i = 0; i < nch; ++i) {
        if (inside(i)) {
            const u32x4 p = piece(i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = Piece<T>::get(p, e) - mean[e];
                f[0][e] = fmaf(d, d, f[0][e]);
            }
        }
    }
    strip_total<V, 1, NT>(f, red, tot[1]);
#pragma unroll
    for (int e = 0; e < V; ++e) rstd[e] = 1.0f / sqrtf(tot[1][tl * V + e] * a.inv_c + a.eps);
#pragma unroll NCH > 0 ? NCH : 1
    for (int i = 0; i < nch; ++i) {
        const int c = i * R + cr;
        if (inside(i)) {
            const u32x4 p = piece(i);
            const float g = (float)static_cast<const T*>(a.gamma)[c];
            const float b = a.beta ? (float)static_cast<const T*>(a.beta)[c] : 0.0f;
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = fmaf((Piece<T>::get(p, e) - mean[e]) * rstd[e], g, b);
            store_piece<T>(at_bytes(y, off_y(i)), o, n, !EDGE);
        }
    }
    if (a.mean && cr == 0) {
        const int at = bi * a.S + first + tl * V;   // below b S
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (!EDGE || e < n) {
                a.mean[at + e] = mean[e];
                a.rstd[at + e] = rstd[e];
            }
    }
}

// Sum over the TL token lanes of a channel, in each of them.
__device__ __forceinline__ float token_sum(float v) {
    v += dpp<kQuadXor1>(v);
    v += dpp<kQuadXor2>(v);
    return v;
}

// A workgroup takes strips in turn. While it writes a strip's dx piece by piece, each
// register that becomes free takes the next strip's piece: the loads of one strip run under
// the arithmetic of the one before, with no registers of their own. Loads return in order,
// so nothing else is loaded in between: gamma stays in registers, and a strip's statistics
// are fetched ahead of its pieces.
template <typename T, int NCH, int NT, bool SHIFT, bool EDGE>
__global__ __launch_bounds__(NT) void layer_norm_strips_grad_kernel(NormArgs a) {
    static_assert(!EDGE || NCH == 0, "pieces that end with the slab are not held");
    constexpr int V = Piece<T>::V, R = NT / TL, TT = TL * V, HOLD = NCH > 0 ? NCH : 1;
    __shared__ float red[NT / 64 * 2 * TT];
    __shared__ float tot[2][TT];
    __shared__ float stats[2][TT];
    const int tl = threadIdx.x % TL, cr = threadIdx.x / TL;
    const int nch = NCH > 0 ? NCH : (a.C + R - 1) / R;
    float* out = a.partial + (int64_t)blockIdx.x * 2 * a.C;
    float gamma[HOLD], dg[HOLD], db[HOLD];
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
        gamma[i] = NCH > 0 && i * R + cr < a.C ? (float)static_cast<const T*>(a.gamma)[i * R + cr] : 0.0f;
        dg[i] = db[i] = 0.0f;
    }
    using Off = Offset<NCH>;
    const Off lane_x = ((Off)cr * (Off)a.x_sc + tl * V) * sizeof(T), lane_d = ((Off)cr * (Off)a.S + tl * V) * sizeof(T);
    const Off step_x = (Off)R * (Off)a.x_sc * sizeof(T), step_d = (Off)R * (Off)a.S * sizeof(T);
    const auto off_x = [&](int i) { return from_here(lane_x) + (Off)i * step_x; };
    const auto off_d = [&](int i) { return from_here(lane_d) + (Off)i * step_d; };
    int bi, first, twice, n = V;
    const T* x;
    int64_t dense;
    float stat = 0.0f;
    const auto go_to = [&](int strip) {
        strip_tokens<TT, EDGE>(a, strip, bi, first, twice);
        if (EDGE) n = a.S - first - tl * V;
        x = static_cast<const T*>(a.x) + (int64_t)bi * a.x_sb + first;
        dense = (int64_t)bi * a.C * a.S + first;
        // tokens past S: mean = rstd = 0 and dy = 0, so they add nothing
        const int t = threadIdx.x % TT;
        if (threadIdx.x < 2 * TT && (!EDGE || first + t < a.S))
            stat = (threadIdx.x < TT ? a.mean : a.rstd)[bi * a.S + first + t];   // below b S
    };
    const auto inside = [&](int i) { return ((NCH > 0 && i < NCH - 1) || i * R + cr < a.C) && (!EDGE || n > 0); };
    const auto load_x = [&](int i) {
        return inside(i) ? load_piece(at_bytes(x, off_x(i)), n, !EDGE) : u32x4{0, 0, 0, 0};
    };
    const auto load_d = [&](int i) {
        return inside(i) ? load_piece(at_bytes(static_cast<const T*>(a.dy) + dense, off_d(i)), n, !EDGE) : u32x4{0, 0, 0, 0};
    };
    u32x4 hx[HOLD], hd[HOLD];
    const int strip0 = strip_of(blockIdx.x, gridDim.x);
    go_to(strip0);   // there are no more workgroups than strips
    if constexpr (NCH > 0) {
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
            hx[i] = load_x(i);
            hd[i] = load_d(i);
        }
    }
    for (int strip = strip0; strip < a.all_strips; strip += gridDim.x) {
        if (threadIdx.x < 2 * TT) (&stats[0][0])[threadIdx.x] = stat;
        __syncthreads();
        float mean[V], rstd[V], f[2][V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            mean[e] = stats[0][tl * V + e];
            rstd[e] = stats[1][tl * V + e];
            f[0][e] = f[1][e] = 0.0f;
        }
#pragma unroll NCH > 0 ? NCH : 1
        for (int i = 0; i < nch; ++i) {
            const int c = i * R + cr;
            float sg = 0.0f, sb = 0.0f;
            if ((NCH > 0 && i < NCH - 1) || c < a.C) {
                const u32x4 px = NCH > 0 ? hx[NCH > 0 ? i : 0] : load_x(i), pd = NCH > 0 ? hd[NCH > 0 ? i : 0] : load_d(i);
                const float g = NCH > 0 ? gamma[NCH > 0 ? i : 0] : (float)static_cast<const T*>(a.gamma)[c];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float d = Piece<T>::get(pd, e);
                    const float xh = (Piece<T>::get(px, e) - mean[e]) * rstd[e], gd = d * g;
                    f[0][e] += gd;
                    f[1][e] = fmaf(gd, xh, f[1][e]);
                    if (!SHIFT || tl * V + e >= twice) {
                        sg = fmaf(d, xh, sg);
                        sb += d;
                    }
                }
            }
            if constexpr (NCH > 0) {
                dg[i] += sg;
                db[i] += sb;
                settle(dg[i]);
                settle(db[i]);
                __builtin_amdgcn_sched_barrier(0);
            } else {
                // this thread alone writes the channel's sums of this workgroup
                sg = token_sum(sg);
                sb = token_sum(sb);
                if (tl == 0 && c < a.C) {
                    out[c] = strip == strip0 ? sg : out[c] + sg;
                    out[a.C + c] = strip == strip0 ? sb : out[a.C + c] + sb;
                }
            }
        }
        strip_total<V, 2, NT>(f, red, tot[0]);
        // dx = rstd (d gamma - c1 - xhat c2) = d gamma rstd + (x - mean) t2 + t1
        float t1[V], t2[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            t1[e] = -rstd[e] * (tot[0][tl * V + e] * a.inv_c);
            t2[e] = -rstd[e] * (rstd[e] * (tot[1][tl * V + e] * a.inv_c));
        }
        T* dx = static_cast<T*>(a.y) + dense;
        const bool more = strip + (int)gridDim.x < a.all_strips;
        if (NCH > 0 && more) go_to(strip + gridDim.x);
#pragma unroll NCH > 0 ? NCH : 1
        for (int i = 0; i < nch; ++i) {
            if constexpr (NCH > 0) {
                unpack_again(hx[i]);
                unpack_again(hd[i]);
            }
            if (inside(i)) {
                const u32x4 px = NCH > 0 ? hx[NCH > 0 ? i : 0] : load_x(i), pd = NCH > 0 ? hd[NCH > 0 ? i : 0] : load_d(i);
                const float g = NCH > 0 ? gamma[NCH > 0 ? i : 0] : (float)static_cast<const T*>(a.gamma)[i * R + cr];
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o[e] = fmaf(Piece<T>::get(px, e) - mean[e], t2[e], fmaf(Piece<T>::get(pd, e) * g, rstd[e], t1[e]));
                store_piece<T>(at_bytes(dx, off_d(i)), o, n, !EDGE);
                if constexpr (NCH > 0) {
                    if (more) {
                        hx[i] = load_x(i);
                        hd[i] = load_d(i);
                    }
                }
            }
            // the refill takes the registers just freed: no load moves up to where it would need others
            __builtin_amdgcn_sched_barrier(0);
        }
        if (NCH == 0 && more) go_to(strip + gridDim.x);
        // the next strip's statistics and totals are written where every thread has read this
        // one's: stats before the totals' barriers, totals before the next statistics'
    }
    if constexpr (NCH > 0) {
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
            const int c = i * R + cr;
            const float sg = token_sum(dg[i]), sb = token_sum(db[i]);
            if (tl == 0 && c < a.C) {
                out[c] = sg;
                out[a.C + c] = sb;
            }
        }
    }
}

// ------------------------------------------------------------------ dgamma and dbeta
// Adds the workgroups' sums: 32 columns of [2, C] a workgroup, 32 threads a column.
template <typename T>
__global__ __launch_bounds__(1024) void layer_norm_columns_kernel(const float* partial, T* dgamma, T* dbeta, int C,
                                                                  int parts) {
    __shared__ double red[32][33];
    // rows of kMostBlocks; the last workgroups may be past the columns, 2^30 + 2^25 at most
    const int col = (int)(blockIdx.y * gridDim.x + blockIdx.x) * 32 + (int)(threadIdx.x & 31), r = threadIdx.x >> 5;
    double s = 0.0;
    if (col < 2 * C) {
        int p = r;
        for (; p + 7 * 32 < parts; p += 8 * 32) {   // 8 loads in flight
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = partial[(int64_t)(p + k * 32) * 2 * C + col];
#pragma unroll
            for (int k = 0; k < 8; ++k) s += (double)v[k];
        }
        for (; p < parts; p += 32) s += (double)partial[(int64_t)p * 2 * C + col];
    }
    red[r][threadIdx.x & 31] = s;
    __syncthreads();
    if (r == 0 && col < 2 * C) {
#pragma unroll
        for (int k = 1; k < 32; ++k) s += red[k][threadIdx.x];
        if (col < C)
            dgamma[col] = (T)(float)s;
        else if (dbeta)
            dbeta[col - C] = (T)(float)s;
    }
}

// ------------------------------------------------------------------ plans
constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;
// Loops over tokens and strips step by up to 2^22 past the last (kMostBlocks workgroups of 4
// rows) in 32 bits, and dgamma and dbeta are 2 C columns in 32 bits.
constexpr int64_t kMostTokens = (int64_t(1) << 31) - (int64_t(1) << 23), kMostChannels = int64_t(1) << 29;
constexpr int kMostBlocks = 1 << 20;   // along a grid's dimension, of up to 1024 threads: fewer than 2^32

struct Derived {
    int64_t S = 0, M = 0, C = 0, sb = 0, ss = 0, sc = 0, x_span = 0;
    bool first = false, edge = false;   // channels-first; its slabs shorter than a strip
    int esize = 0, V = 0;
    int tpr = 0, nt = 0, nch = 0;   // threads a row or strip, pieces a thread
    int parts = 0;                  // backward: workgroups, and rows of the workspace
};

int64_t mul_cap(int64_t a, int64_t b) {
    const int64_t lim = int64_t(1) << 60;
    if (a < 0 || b < 0) return -1;
    if (a == 0 || b == 0) return 0;
    return a > lim / b ? -1 : a * b;
}

int at_least(int n, std::initializer_list<int> among) {
    for (int k : among)
        if (k >= n) return k;
    return 0;
}

int check(const layer_norm_desc* d, Derived* out) {
    if (!d) return FUSED_PROJ_EINVAL;
    if (d->dtype != FUSED_PROJ_BF16 && d->dtype != FUSED_PROJ_F32) return FUSED_PROJ_EINVAL;
    if (d->x_layout != FUSED_PROJ_X_CHANNELS_FIRST && d->x_layout != FUSED_PROJ_X_TOKENS_LAST) return FUSED_PROJ_EINVAL;
    if (d->batch < 0 || d->channels < 1) return FUSED_PROJ_EINVAL;
    if (d->x_layout == FUSED_PROJ_X_TOKENS_LAST ? d->n_spatial != 1 : (d->n_spatial < 1 || d->n_spatial > 3))
        return FUSED_PROJ_EINVAL;
    if (d->x_stride_batch < 0 || d->x_stride_channel < 0) return FUSED_PROJ_EINVAL;
    for (int i = 0; i < d->n_spatial; ++i)
        if (d->spatial[i] < 0 || d->x_stride_spatial[i] < 0) return FUSED_PROJ_EINVAL;
    if (d->has_bias != 0 && d->has_bias != 1) return FUSED_PROJ_EINVAL;
    if (!(d->eps >= 0.0) || !std::isfinite((float)d->eps)) return FUSED_PROJ_EINVAL;
    Derived r;
    r.esize = d->dtype == FUSED_PROJ_BF16 ? 2 : 4;
    r.V = 16 / r.esize;
    r.C = d->channels;
    r.first = d->x_layout == FUSED_PROJ_X_CHANNELS_FIRST;
    r.S = 1;
    for (int i = 0; i < d->n_spatial; ++i) {
        r.S = mul_cap(r.S, d->spatial[i]);
        if (r.S < 0) return FUSED_PROJ_EUNSUPPORTED;
    }
    r.M = mul_cap(d->batch, r.S);
    if (r.M < 0 || r.M > kMostTokens || r.S > kMostTokens || r.C > kMostChannels || mul_cap(r.M, r.C) < 0)
        return FUSED_PROJ_EUNSUPPORTED;
    r.sb = d->x_stride_batch;
    r.sc = d->x_stride_channel;
    if (!r.first) {
        r.ss = d->x_stride_spatial[0];
        if (r.M > 0 && r.C > 1 && r.sc != 1) return FUSED_PROJ_EUNSUPPORTED;
        r.sc = 1;
        if (r.C > 32768) return FUSED_PROJ_EUNSUPPORTED;
    } else {
        int64_t expect = 1;
        for (int i = d->n_spatial - 1; i >= 0; --i) {
            if (r.M > 0 && d->spatial[i] > 1 && d->x_stride_spatial[i] != expect) return FUSED_PROJ_EUNSUPPORTED;
            expect *= d->spatial[i];
        }
        r.ss = 1;
    }
    if (r.M > 0) {
        const int64_t a = mul_cap(d->batch - 1, r.sb), b = mul_cap(r.S - 1, r.ss), c = mul_cap(r.C - 1, r.sc);
        if (a < 0 || b < 0 || c < 0) return FUSED_PROJ_EUNSUPPORTED;
        r.x_span = a + b + c + 1;
    }
    const int V = r.V, C = (int)r.C;
    if (!r.first) {
        // A wave a row while the row fits 4 pieces a lane (no barriers); else a workgroup.
        r.tpr = C <= 64 * V * 4 ? 64 : C <= 256 * V * 4 ? 256 : 1024;
        const int need = (C + r.tpr * V - 1) / (r.tpr * V);
        r.nch = r.tpr == 1024 ? at_least(need, {2, 4, 8}) : at_least(need, {1, 2, 3, 4});
        const int rpb = r.tpr < 512 ? 512 / r.tpr : 1;
        const int64_t want = (r.M + rpb - 1) / rpb;
        r.parts = (int)(want < 512 ? want : 512);
    } else {
        // as many threads as leave each 6 pieces or fewer
        r.nt = C <= 64 * 6 ? 256 : C <= 128 * 6 ? 512 : 1024;
        const int need = (C + r.nt / 4 - 1) / (r.nt / 4);
        r.nch = at_least(need, {1, 2, 3, 4, 5, 6});
        // held strips: slabs of a strip or more, offsets within a slab in 32 bits of bytes
        r.edge = r.S < TL * V;
        const int64_t reach = mul_cap(r.C, r.sc > r.S ? r.sc : r.S);
        if (r.edge || reach < 0 || reach * r.esize > 2 * kMaxIndex) r.nch = 0;
        if (r.nch == 0) r.nt = 1024;
        const int64_t strips = mul_cap(d->batch, (r.S + TL * V - 1) / (TL * V)), turn = 256 * (1024 / r.nt);
        r.parts = (int)(strips < turn ? strips : turn);
    }
    if (out) *out = r;
    return FUSED_PROJ_OK;
}

struct Range {
    uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes}; }
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }
bool misaligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1); }

}  // namespace

struct layer_norm_plan {
    layer_norm_desc d;
    Derived r;
    int device = -1;
};

namespace {

int hip_status(hipError_t e) {
    if (e == hipSuccess) return FUSED_PROJ_OK;
    fp::set_last_hip_error(e);
    return FUSED_PROJ_EHIP;
}

int on_device(const layer_norm_plan* h) {
    int dev = -1;
    const int rc = hip_status(hipGetDevice(&dev));
    if (rc) return rc;
    return dev == h->device ? FUSED_PROJ_OK : FUSED_PROJ_EINVAL;
}

NormArgs base_args(const layer_norm_plan* h, const void* x, const void* gamma) {
    const Derived& r = h->r;
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.gamma = gamma;
    a.x_sb = r.sb;
    a.x_ss = r.ss;
    a.x_sc = r.sc;
    a.M = (int32_t)r.M;
    a.S = (int32_t)r.S;
    a.C = (int32_t)r.C;
    a.inv_c = (float)(1.0 / (double)r.C);
    a.eps = (float)h->d.eps;
    if (r.first) {
        a.strips = (int32_t)((r.S + TL * r.V - 1) / (TL * r.V));
        a.all_strips = (int32_t)(h->d.batch * a.strips);
        a.div_s = fp::make_fastdiv_u31((uint32_t)a.strips);
    } else {
        a.div_s = fp::make_fastdiv_u31((uint32_t)r.S);
    }
    return a;
}

dim3 grid_of(int64_t blocks) {
    const unsigned x = (unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks);
    return dim3(x, (unsigned)((blocks + x - 1) / x));
}
void launch(void (*kernel)(NormArgs), int64_t grid, int block, const NormArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(kernel, grid_of(grid), dim3(block), 0, st, a);
}

template <typename T, bool TAIL>
void launch_rows(const Derived& r, const NormArgs& a, bool grad, hipStream_t st) {
    const int tpr = r.tpr, nch = r.nch;
    const int block = tpr < (grad ? 512 : 256) ? (grad ? 512 : 256) : tpr, rpb = block / tpr;
    const int64_t want = (r.M + rpb - 1) / rpb, grid = grad ? r.parts : want < kMostBlocks ? want : kMostBlocks;
#define LN_CASE(N, TPR)                                                                         \
    if (tpr == TPR && nch == N)                                                                 \
        return launch(grad ? layer_norm_rows_grad_kernel<T, N, TPR, TAIL> : layer_norm_rows_kernel<T, N, TPR, TAIL>, \
                      grid, block, a, st);
    LN_CASE(1, 64) LN_CASE(2, 64) LN_CASE(3, 64) LN_CASE(4, 64)
    LN_CASE(2, 256) LN_CASE(3, 256) LN_CASE(4, 256)
    LN_CASE(2, 1024) LN_CASE(4, 1024)
    if constexpr (sizeof(T) == 4) LN_CASE(8, 1024)
#undef LN_CASE
}

template <typename T>
void launch_strips(const Derived& r, const NormArgs& a, bool grad, hipStream_t st) {
    const int64_t grid = grad ? r.parts : a.all_strips;
    const bool shift = r.S % (TL * Piece<T>::V) != 0;
    if (r.edge)
        return launch(grad ? layer_norm_strips_grad_kernel<T, 0, 1024, false, true> : layer_norm_strips_kernel<T, 0, 1024, true>,
                      grid, 1024, a, st);
#define LN_CASE(N, NT)                                                                                   \
    if (r.nt == NT && r.nch == N)                                                                        \
        return launch(!grad   ? layer_norm_strips_kernel<T, N, NT, false>                             \
                      : shift ? layer_norm_strips_grad_kernel<T, N, NT, true, false>                  \
                              : layer_norm_strips_grad_kernel<T, N, NT, false, false>,                \
                      grid, NT, a, st);
    LN_CASE(1, 256) LN_CASE(2, 256) LN_CASE(3, 256) LN_CASE(4, 256) LN_CASE(5, 256) LN_CASE(6, 256)
    LN_CASE(4, 512) LN_CASE(5, 512) LN_CASE(6, 512)
    LN_CASE(4, 1024) LN_CASE(5, 1024) LN_CASE(6, 1024) LN_CASE(0, 1024)
#undef LN_CASE
}

template <typename T>
void launch_any(const Derived& r, const NormArgs& a, bool grad, hipStream_t st) {
    if (r.first)
        launch_strips<T>(r, a, grad, st);
    else if (r.C % r.V != 0)   // the last piece ends past the row
        launch_rows<T, true>(r, a, grad, st);
    else
        launch_rows<T, false>(r, a, grad, st);
}

}  // namespace

extern "C" {

int layer_norm_validate(const layer_norm_desc* desc) { return check(desc, nullptr); }

int layer_norm_create(const layer_norm_desc* desc, layer_norm_t* out) {
    if (!out) return FUSED_PROJ_EINVAL;
    *out = nullptr;
    Derived r;
    int rc = check(desc, &r);
    if (rc) return rc;
    layer_norm_plan* h = new (std::nothrow) layer_norm_plan();
    if (!h) return FUSED_PROJ_EHIP;
    h->d = *desc;
    h->r = r;
    rc = hip_status(hipGetDevice(&h->device));
    if (rc) {
        delete h;
        return rc;
    }
    *out = h;
    return FUSED_PROJ_OK;
}

int layer_norm_run(layer_norm_t h, const void* x, const void* gamma, const void* beta, void* y, void* stats,
                   void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    const Derived& r = h->r;
    if (r.M == 0) return FUSED_PROJ_OK;
    const bool bias = h->d.has_bias;
    if (!x || !gamma || (bias && !beta) || !y) return FUSED_PROJ_EINVAL;
    for (const void* p : {x, gamma, bias ? beta : gamma, (const void*)y})
        if (misaligned(p, r.esize)) return FUSED_PROJ_EALIGN;
    if (misaligned(stats, 4)) return FUSED_PROJ_EALIGN;
    const Range ins[3] = {range(x, r.x_span * r.esize), range(gamma, r.C * r.esize),
                          range(bias ? beta : gamma, r.C * r.esize)};
    const Range ry = range(y, r.M * r.C * r.esize), rs = range(stats, stats ? r.M * 8 : 0);
    for (const Range& i : ins)
        if (overlap(ry, i) || overlap(rs, i)) return FUSED_PROJ_EALIAS;
    if (overlap(ry, rs)) return FUSED_PROJ_EALIAS;
    const int rc = on_device(h);
    if (rc) return rc;
    NormArgs a = base_args(h, x, gamma);
    a.beta = bias ? beta : nullptr;
    a.y = y;
    a.mean = static_cast<float*>(stats);
    a.rstd = stats ? a.mean + r.M : nullptr;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (h->d.dtype == FUSED_PROJ_BF16)
        launch_any<__bf16>(r, a, false, st);
    else
        launch_any<float>(r, a, false, st);
    return hip_status(hipGetLastError());
}

int layer_norm_backward_workspace_size(layer_norm_t h, size_t* bytes) {
    if (!h || !bytes) return FUSED_PROJ_EINVAL;
    *bytes = (size_t)h->r.parts * 2 * (size_t)h->r.C * sizeof(float);
    return FUSED_PROJ_OK;
}

int layer_norm_backward(layer_norm_t h, const void* x, const void* gamma, const void* stats, const void* dy, void* dx,
                        void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes, void* stream) {
    if (!h) return FUSED_PROJ_EINVAL;
    const Derived& r = h->r;
    const bool bias = h->d.has_bias;
    if (!dgamma || (bias && !dbeta)) return FUSED_PROJ_EINVAL;
    const size_t need = (size_t)r.parts * 2 * (size_t)r.C * sizeof(float);
    if (r.M > 0) {
        if (!x || !gamma || !stats || !dy || !dx || !workspace || workspace_bytes < need) return FUSED_PROJ_EINVAL;
        for (const void* p : {x, gamma, dy, (const void*)dx})
            if (misaligned(p, r.esize)) return FUSED_PROJ_EALIGN;
        if (misaligned(stats, 4) || misaligned(workspace, 16)) return FUSED_PROJ_EALIGN;
    }
    for (const void* p : {(const void*)dgamma, bias ? (const void*)dbeta : (const void*)dgamma})
        if (misaligned(p, r.esize)) return FUSED_PROJ_EALIGN;
    const int64_t cb = r.C * r.esize, nb = r.M * r.C * r.esize;
    const bool any = r.M > 0;
    const Range ins[4] = {range(x, any ? r.x_span * r.esize : 0), range(gamma, any ? cb : 0),
                          range(stats, any ? r.M * 8 : 0), range(dy, nb)};
    const Range outs[4] = {range(dx, nb), range(dgamma, cb), range(dbeta, bias ? cb : 0),
                           range(workspace, any ? (int64_t)need : 0)};
    for (int i = 0; i < 4; ++i) {
        for (const Range& in : ins)
            if (overlap(outs[i], in)) return FUSED_PROJ_EALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return FUSED_PROJ_EALIAS;
    }
    const int rc = on_device(h);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (r.M > 0) {
        NormArgs a = base_args(h, x, gamma);
        a.dy = dy;
        a.y = dx;
        a.mean = const_cast<float*>(static_cast<const float*>(stats));
        a.rstd = a.mean + r.M;
        a.partial = static_cast<float*>(workspace);
        if (h->d.dtype == FUSED_PROJ_BF16)
            launch_any<__bf16>(r, a, true, st);
        else
            launch_any<float>(r, a, true, st);
        const int rc2 = hip_status(hipGetLastError());
        if (rc2) return rc2;
    }
    // with no tokens there are no parts, and the sums are 0
    const dim3 grid = grid_of((2 * r.C + 31) / 32);
    if (h->d.dtype == FUSED_PROJ_BF16)
        hipLaunchKernelGGL((layer_norm_columns_kernel<__bf16>), grid, dim3(1024), 0, st,
                           static_cast<const float*>(workspace), static_cast<__bf16*>(dgamma),
                           static_cast<__bf16*>(bias ? dbeta : nullptr), (int)r.C, r.parts);
    else
        hipLaunchKernelGGL((layer_norm_columns_kernel<float>), grid, dim3(1024), 0, st,
                           static_cast<const float*>(workspace), static_cast<float*>(dgamma),
                           static_cast<float*>(bias ? dbeta : nullptr), (int)r.C, r.parts);
    return hip_status(hipGetLastError());
}

int layer_norm_destroy(layer_norm_t h) {
    delete h;
    return FUSED_PROJ_OK;
}

}  // extern "C"
