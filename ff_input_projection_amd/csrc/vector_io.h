// 16-byte pieces of bf16 or fp32 rows, and sums across the lanes of a wave (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace fp {
namespace dev {

// T's values as 16-byte pieces of V. Global loads and stores of 16 bytes need no more than
// the element's alignment here (unaligned access is on for this target), so rows of any
// length and any start are read and written with them.
template <typename T>
struct Piece;
template <>
struct Piece<__bf16> {
    static constexpr int V = 8;
    static __device__ __forceinline__ float get(const u32x4& r, int e) {
        const uint32_t w = r[e >> 1];
        return __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
    static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
        bf16x8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (__bf16)f[e];
        return __builtin_bit_cast(u32x4, o);
    }
};
template <>
struct Piece<float> {
    static constexpr int V = 4;
    static __device__ __forceinline__ float get(const u32x4& r, int e) { return __uint_as_float(r[e]); }
    static __device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
        return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};

// The first n of V values at p, the rest 0; with `whole`, all V in one load.
template <typename T>
__device__ __forceinline__ u32x4 load_piece(const T* p, int n, bool whole) {
    constexpr int V = Piece<T>::V;
    u32x4 r = {0, 0, 0, 0};
    if (whole || n >= V) {
        __builtin_memcpy(&r, p, 16);
    } else {
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = e < n ? (float)p[e] : 0.0f;
        r = Piece<T>::pack(f);   // exact: the values are T's
    }
    return r;
}
// The first n of V values to p (all of them with `whole`); the values behind them stay as
// they were.
template <typename T>
__device__ __forceinline__ void store_piece(T* p, const float (&f)[Piece<T>::V], int n, bool whole) {
    constexpr int V = Piece<T>::V;
    if (whole || n >= V) {
        const u32x4 r = Piece<T>::pack(f);
        __builtin_memcpy(p, &r, 16);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < n) p[e] = (T)f[e];
    }
}

// Makes a held piece opaque: the compiler unpacks it again for the next use instead of
// keeping its V unpacked values in registers since the last one.
__device__ __forceinline__ void unpack_again(u32x4& r) { asm volatile("" : "+v"(r)); }

// Makes the compiler compute x here: a sum that is needed only behind a loop would else be
// added up at the loop's end, its terms kept in registers until there.
__device__ __forceinline__ void settle(float& x) { asm volatile("" : "+v"(x)); }
// The same value, computed from here on: what depends on it is not moved out of a loop (an
// offset widened to 64 bits there would take two registers, and the short form of a load).
__device__ __forceinline__ uint32_t from_here(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}
__device__ __forceinline__ uint64_t from_here(uint64_t x) { return x; }

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kRowRor8 = 0x128;

// a' = {a's lower half, b's lower half} and b' = {a's upper, b's upper}, halves of 32 lanes;
// a' + b' then holds a's sum over lane bit 5 in the lower half and b's in the upper one.
__device__ __forceinline__ float swap_sum32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The same over lane bit 4: rows of 16 lanes; odd rows end with b's sum.
__device__ __forceinline__ float swap_sum16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Sum over all 64 lanes, the same bits in each.
__device__ __forceinline__ float wave_sum(float x) {
    x += dpp<kQuadXor1>(x);
    x += dpp<kQuadXor2>(x);
    x += dpp<kHalfMirror>(x);   // both quads of each 8 lanes hold one value each: mirrored is the other quad
    x += dpp<kRowRor8>(x);
    x = swap_sum16(x, x);
    return swap_sum32(x, x);
}

}  // namespace dev
}  // namespace fp
