// Device helpers shared by the token cache's kernels: lane exchanges and the
// Hadamard transform of rows held 8 features to a lane.
#pragma once
#include "cache.h"
#include "dev_common.h"

namespace jolt {

constexpr int kDppQuadReverse = 0x1B;   // quad_perm [3, 2, 1, 0]

// a lane move inside rows of 16 whose source lane always exists (so no old value
// is kept for it)
template <int Ctrl>
__device__ __forceinline__ float row_move(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), Ctrl, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_xor1(float v) { return row_move<kDppXor1>(v); }
__device__ __forceinline__ float lane_xor2(float v) { return row_move<kDppXor2>(v); }
// i ^ 7 (half mirror), then i ^ 3
__device__ __forceinline__ float lane_xor4(float v) { return row_move<kDppQuadReverse>(row_move<kDppHalfMirror>(v)); }
// i ^ 15 (row mirror), then i ^ 7
__device__ __forceinline__ float lane_xor8(float v) { return row_move<kDppHalfMirror>(row_move<kDppMirror>(v)); }

template <int X>
__device__ __forceinline__ float lane_xor(float v) {
    static_assert(X == 1 || X == 2 || X == 4 || X == 8, "within a row of 16 lanes");
    if constexpr (X == 1) return lane_xor1(v);
    else if constexpr (X == 2) return lane_xor2(v);
    else if constexpr (X == 4) return lane_xor4(v);
    else return lane_xor8(v);
}
template <int X>
__device__ __forceinline__ double lane_xor(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const float lo = lane_xor<X>(__uint_as_float((uint32_t)u));
    const float hi = lane_xor<X>(__uint_as_float((uint32_t)(u >> 32)));
    return __builtin_bit_cast(double, (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32));
}
// largest value over aligned groups of N lanes (N = 8, 16), as unsigned integers
template <int N>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
    v = max(v, __float_as_uint(lane_xor<1>(__uint_as_float(v))));
    v = max(v, __float_as_uint(lane_xor<2>(__uint_as_float(v))));
    v = max(v, __float_as_uint(lane_xor<4>(__uint_as_float(v))));
    if constexpr (N == 16) v = max(v, __float_as_uint(lane_xor<8>(__uint_as_float(v))));
    return v;
}

template <int X, typename T>
__device__ __forceinline__ void fwht_lanes(T (&x)[8], int j) {
    const T s = (j & X) ? T(-1) : T(1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const T o = lane_xor<X>(x[e]);
        if constexpr (sizeof(T) == 8) x[e] = fma(x[e], s, o);      // o + x or o - x, rounded once
        else x[e] = fmaf(x[e], s, o);
    }
}
// Unscaled Sylvester Hadamard transform of rows of D features, lane j of the
// row's D/8 consecutive lanes holding features 8 j .. 8 j + 7.  Every lane of
// the wave must call it.
template <int D, typename T>
__device__ __forceinline__ void fwht_row(T (&x)[8], int j) {
#pragma unroll
    for (int h = 1; h < 8; h *= 2)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!(e & h)) {
                const T a = x[e], b = x[e + h];
                x[e] = a + b;
                x[e + h] = a - b;
            }
    fwht_lanes<1>(x, j);
    fwht_lanes<2>(x, j);
    fwht_lanes<4>(x, j);
    if constexpr (D == 128) fwht_lanes<8>(x, j);
}

// sign bits of features 8 j .. 8 j + 7
__device__ __forceinline__ uint32_t sign_byte(const uint32_t (&s)[4], int j) {
    const uint32_t lo = (j & 4) ? s[1] : s[0], hi = (j & 4) ? s[3] : s[2];
    return (((j & 8) ? hi : lo) >> (8 * (j & 3))) & 0xFFu;
}
__device__ __forceinline__ double flip(double v, bool neg) { return neg ? -v : v; }
__device__ __forceinline__ float flip(float v, bool neg) { return neg ? -v : v; }

// nibble of member e of a 4-bit unit
__device__ __forceinline__ constexpr int nibble_of(int e) { return 4 * (e / 2 + 4 * (e % 2)); }

// a unit of 8 codes as bf16 (4 bits: 128 + code, 8 bits: code)
template <int BITS>
__device__ __forceinline__ bf16x8 unit_bf16(const uint32_t *w) {
    uint32_t r[4];
    if constexpr (BITS == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = ((w[0] >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = w[i >> 1] >> (16 * (i & 1));
            const uint32_t lo = __float_as_uint((float)(v & 255u)), hi = __float_as_uint((float)((v >> 8) & 255u));
            r[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);       // the upper halves: integers < 256 fit bf16
        }
    }
    const uint4 q = make_uint4(r[0], r[1], r[2], r[3]);
    return __builtin_bit_cast(bf16x8, q);
}

// N dwords from a 16-byte (N = 4, 8, ...) or 8-byte (N = 2) aligned address
template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    }
}

}  // namespace jolt
