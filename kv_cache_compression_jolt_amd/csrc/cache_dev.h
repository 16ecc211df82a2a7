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
    const bool up = j & X;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const T o = lane_xor<X>(x[e]);
        x[e] = up ? o - x[e] : x[e] + o;
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

}  // namespace jolt
