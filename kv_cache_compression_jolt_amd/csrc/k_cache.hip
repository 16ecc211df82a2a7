// Token cache: writing rows (rotate, quantize, pack), reading them back, and
// moving accepted drafted tokens.  Page layout: libjolt.h.
//
// All three work on (sequence, block of 8 tokens, head): the 8 tokens that
// share the V units, so that a workgroup owns every unit it rewrites and no
// two workgroups touch one word.
#include "cache.h"
#include "cache_dev.h"
#include "jolt_internal.h"
#include "ktimer.h"

namespace jolt {

namespace {

template <typename T> __device__ __forceinline__ void load8(const T *p, float (&x)[8]);
template <> __device__ __forceinline__ void load8<uint16_t>(const uint16_t *p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <> __device__ __forceinline__ void load8<float>(const float *p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// store 8 values, the sign of value e changed where bit e of `neg` is set
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&x)[8], uint32_t neg);
template <> __device__ __forceinline__ void store8<uint16_t>(uint16_t *p, const float (&x)[8], uint32_t neg) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = neg >> (2 * i);
        w[i] = bf16_pair(x[2 * i], x[2 * i + 1]) ^ (((two & 1u) << 15) | ((two & 2u) << 30));
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store8<float>(float *p, const float (&x)[8], uint32_t neg) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(__float_as_uint(x[e]) ^ (((neg >> e) & 1u) << 31));
    reinterpret_cast<float4 *>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}

// 8 codes as one unit: 8 bytes, or the 32-bit word of a 4-bit cache (in .x)
template <int BITS>
__device__ __forceinline__ uint2 pack_unit(const uint32_t (&u)[8]) {
    if constexpr (BITS == 4) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= u[e] << nibble_of(e);
        return make_uint2(w, 0);
    } else {
        return make_uint2(u[0] | (u[1] << 8) | (u[2] << 16) | (u[3] << 24),
                          u[4] | (u[5] << 8) | (u[6] << 16) | (u[7] << 24));
    }
}
template <int BITS>
__device__ __forceinline__ uint32_t unit_code(uint2 w, int e) {
    if constexpr (BITS == 4) return (w.x >> nibble_of(e)) & 15u;
    else return ((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 255u;
}
template <int BITS>
__device__ __forceinline__ uint2 load_unit(const uint8_t *codes, int64_t unit) {
    if constexpr (BITS == 4) return make_uint2(reinterpret_cast<const uint32_t *>(codes)[unit], 0);
    else return reinterpret_cast<const uint2 *>(codes)[unit];
}
template <int BITS>
__device__ __forceinline__ void store_unit(uint8_t *codes, int64_t unit, uint2 w) {
    if constexpr (BITS == 4) reinterpret_cast<uint32_t *>(codes)[unit] = w.x;
    else reinterpret_cast<uint2 *>(codes)[unit] = w;
}
// bits of member e set
template <int BITS>
__device__ __forceinline__ uint2 member_mask(int e) {
    if constexpr (BITS == 4) return make_uint2(15u << nibble_of(e), 0);
    else return e < 4 ? make_uint2(255u << (8 * e), 0) : make_uint2(0, 255u << (8 * (e - 4)));
}

typedef short s16x2 __attribute__((ext_vector_type(2)));

// Workgroups in the order of the dense rows: heads next to each other where a
// token's heads are, token blocks where a head's tokens are.
struct BlockId { int b, blk, h; };
__device__ __forceinline__ BlockId block_id(const CacheRowsArgs &a, int nblk) {
    const uint32_t w = blockIdx.x, H = a.c.H, per = nblk * H;
    const uint32_t in = w % per;
    BlockId r;
    r.b = w / per;
    if (a.k.hs > a.k.ts) {
        r.h = in / nblk;
        r.blk = in % nblk;
    } else {
        r.blk = in / H;
        r.h = in % H;
    }
    return r;
}

// Quantize 8 features of a row (lane j of D/8): the codes, and the group's
// scale bits.  The absolute maximum is taken over the bits as integers, where
// infinities and NaN are above every number, so a row that holds one is seen.
template <int D, int BITS>
__device__ __forceinline__ uint16_t quantize8(const float (&y)[8], uint32_t (&u)[8]) {
    uint32_t am = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) am = max(am, __float_as_uint(y[e]) & 0x7FFFFFFFu);
    am = group_umax<8>(am);
    // the whole row's maximum: every lane takes part in the exchange, before any branch
    uint32_t row_am = am;
    if constexpr (D == 128) row_am = max(am, __float_as_uint(lane_xor<8>(__uint_as_float(am))));
    const bool bad = row_am >= 0x7F800000u;
    constexpr float qmax = (float)((1 << (BITS - 1)) - 1);
    uint16_t sbits = f32_to_bf16(bad ? 0.f : __uint_as_float(am) / qmax);
    if (sbits < 0x0080) sbits = 0;                      // below 2^-126
    const float scale = bf16_to_f32(sbits);
    const float inv = sbits == 0 ? 0.f : 1.0f / scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = bad ? 0.f : fminf(fmaxf(rintf(y[e] * inv), -qmax), qmax);
        u[e] = (uint32_t)((int)q + (1 << (BITS - 1)));
    }
    return bad ? (uint16_t)0x7FC0 : sbits;
}

}  // namespace

// ---------------------------------------------------------------- append
// One workgroup of D threads per (sequence, block of 8 tokens, head): thread
// (row r, lane j) takes features 8 j .. 8 j + 7 of token 8 blk + r.  Its 8 K
// codes are one unit; V codes go through LDS, where thread f then gathers
// feature f of the 8 tokens.  A block that the call only partly covers keeps
// the other tokens' codes (read, merge, write).
//
// The rotation runs in fp64: a bf16 row's +-1 sums of 128 terms are exact there
// (8 + 7 bits, and exponents up to 38 apart), so the one rounding to fp32 and
// with it every code is independent of the order of the butterflies.
template <typename T, int D, int BITS, bool ROT>
__global__ __launch_bounds__(D) void k_cache_append(CacheRowsArgs a, int nblk) {
    const BlockId id = block_id(a, nblk);
    int s0;
    const int n = ragged_rows(a.starts, id.b, a.total, &s0);
    if (n == 0) return;
    const int t0 = a.c.lens[id.b] - n;                   // token of the first row (may lie before 0)
    const int last = t0 + min(n, a.max_rows) - 1, from = max(t0, 0);
    if (last < from) return;
    const int tok8 = ((from >> 3) + id.blk) * 8;
    if (tok8 > last) return;
    const int page = cache_page(a.c, id.b, tok8);
    if (page < 0) return;
    uint8_t *base = a.c.pool + cache_block_offset(a.c, page, id.h);
    const int P = 1 << a.c.page_shift, tin = tok8 & (P - 1);
    const PageLayout pl = page_layout(P, D, BITS);
    const int tid = threadIdx.x, j = tid % (D / 8), r = tid / (D / 8), t = tok8 + r;
    const bool on = t >= from && t <= last;
    const int64_t row = (int64_t)s0 + (t - t0);
    __shared__ __align__(16) uint8_t vc[8][D];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const RowsView &src = kv ? a.v : a.k;
        float x[8];
        if (on) load8(static_cast<const T *>(src.ptr) + row * src.ts + id.h * src.hs + 8 * j, x);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
        }
        if constexpr (ROT) {
            const uint32_t sb = sign_byte(kv ? a.c.sv : a.c.sk, j);
            double y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = flip((double)x[e], (sb >> e) & 1);
            fwht_row<D>(y, j);
            const double isd = D == 128 ? 0.08838834764831845 : 0.125;      // 1 / sqrt(D)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (float)(y[e] * isd);
        }
        uint32_t u[8];
        const uint16_t sbits = quantize8<D, BITS>(x, u);
        if (on && (j & 7) == 0)
            reinterpret_cast<uint16_t *>(base + (kv ? pl.v_scales : pl.k_scales))[(j >> 3) * P + tin + r] = sbits;
        if (kv == 0) {
            if (on) store_unit<BITS>(base, (int64_t)(tin + r) * (D / 8) + (j & 3) * (D / 32) + (j >> 2), pack_unit<BITS>(u));
        } else {
            *reinterpret_cast<uint2 *>(&vc[r][8 * j]) = pack_unit<8>(u);
        }
    }
    __syncthreads();
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = vc[e][tid];
    uint2 w = pack_unit<BITS>(u);
    const int64_t unit = (int64_t)(tin >> 3) * D + tid;
    if (tok8 < from || tok8 + 7 > last) {
        uint2 m = make_uint2(0, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (tok8 + e >= from && tok8 + e <= last) {
                const uint2 me = member_mask<BITS>(e);
                m.x |= me.x;
                m.y |= me.y;
            }
        const uint2 o = load_unit<BITS>(base + pl.v_codes, unit);
        w.x = (w.x & m.x) | (o.x & ~m.x);
        w.y = (w.y & m.y) | (o.y & ~m.y);
    }
    store_unit<BITS>(base + pl.v_codes, unit, w);
}

// ---------------------------------------------------------------- read
// A thread (row r, lane j of D / 8) rebuilds features 8 j .. 8 j + 7 of one token
// of a block of 8, and does so for kReadBlocks blocks at once, so that their
// loads are in flight together.  The rotation of a group of 64 works on the
// unsigned codes as packed 16-bit integers, two features to an instruction (at
// most 64 * 255); their offset only reaches the group's feature 0, as 64 times
// itself.  It is exact, so a value is s0 I0 +- s1 I1 with the scales times isd:
// four roundings.
constexpr int kReadBlocks = 2;

// codes of features 8 j .. 8 j + 7 as 16-bit pairs (2 i, 2 i + 1)
template <int BITS>
__device__ __forceinline__ void key_codes(const uint8_t *codes, int64_t unit, s16x2 (&x)[4]) {
    const uint2 w = load_unit<BITS>(codes, unit);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u;
        if constexpr (BITS == 4) u = (w.x >> (4 * i)) & 0x000F000Fu;
        else u = __builtin_amdgcn_perm(0, i < 2 ? w.x : w.y, (i & 1) ? 0x0C030C02u : 0x0C010C00u);
        x[i] = __builtin_bit_cast(s16x2, u);
    }
}
// member e of the units of 8 consecutive features
template <int BITS>
__device__ __forceinline__ void value_codes(const uint8_t *codes, int64_t unit, int e, s16x2 (&x)[4]) {
    uint32_t w[8];
    if constexpr (BITS == 4) {
        const uint4 *p = reinterpret_cast<const uint4 *>(codes + unit * 4);
        const uint4 a = p[0], b = p[1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(codes + unit * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 a = p[i];
            w[2 * i] = e < 4 ? a.x : a.y;
            w[2 * i + 1] = e < 4 ? a.z : a.w;
        }
    }
    const int sh = BITS == 4 ? nibble_of(e) : 8 * (e & 3);
    constexpr uint32_t mask = BITS == 4 ? 15u : 255u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = __builtin_bit_cast(s16x2, ((w[2 * i] >> sh) & mask) | (((w[2 * i + 1] >> sh) & mask) << 16));
}
template <int X>
__device__ __forceinline__ s16x2 lane_xor_pair(s16x2 v) {
    return __builtin_bit_cast(s16x2, __float_as_uint(lane_xor<X>(__uint_as_float(__builtin_bit_cast(uint32_t, v)))));
}
template <int X>
__device__ __forceinline__ void fwht_pairs_lane(s16x2 (&x)[4], int j) {
    const short s = (j & X) ? -1 : 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const s16x2 o = lane_xor_pair<X>(x[i]);
        x[i] = x[i] * s16x2{s, s} + o;
    }
}
// the 64-point transform over 8 lanes of 8 features each
__device__ __forceinline__ void fwht_pairs(s16x2 (&x)[4], int j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = s16x2{x[i].y, x[i].y} * s16x2{1, -1} + s16x2{x[i].x, x[i].x};
#pragma unroll
    for (int h = 1; h < 4; h *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(i & h)) {
                const s16x2 a = x[i], b = x[i + h];
                x[i] = a + b;
                x[i + h] = a - b;
            }
    fwht_pairs_lane<1>(x, j);
    fwht_pairs_lane<2>(x, j);
    fwht_pairs_lane<4>(x, j);
}

template <typename T, int D, int BITS, bool ROT>
__global__ __launch_bounds__(D) void k_cache_read(CacheRowsArgs a, int nblk) {
    const BlockId id = block_id(a, nblk);
    int s0;
    const int n = min(ragged_rows(a.starts, id.b, a.total, &s0), a.max_rows);
    if (n == 0) return;
    const int64_t f0 = a.first ? a.first[id.b] : 0;
    const int64_t tok8 = ((f0 >> 3) + id.blk * kReadBlocks) * 8;
    if (tok8 >= f0 + n) return;
    const int len = cache_len(a.c, id.b);
    const int tid = threadIdx.x, j = tid % (D / 8), r = tid / (D / 8);
    const int P = 1 << a.c.page_shift;
    const PageLayout pl = page_layout(P, D, BITS);
    constexpr int off = 1 << (BITS - 1);
    s16x2 x[kReadBlocks][2][4];
    float sc[kReadBlocks][2];
#pragma unroll
    for (int i = 0; i < kReadBlocks; ++i) {
        const int64_t t = tok8 + 8 * i;
        const int page = t >= 0 && t < len ? cache_page(a.c, id.b, (int)t) : -1;
        const bool have = page >= 0 && t + r < len;
        const uint8_t *base = a.c.pool + cache_block_offset(a.c, max(page, 0), id.h);
        const int tin = (int)(t & (P - 1));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            sc[i][kv] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][kv][e] = s16x2{off, off};
            if (have)
                sc[i][kv] = bf16_to_f32(reinterpret_cast<const uint16_t *>(base + (kv ? pl.v_scales : pl.k_scales))[(j >> 3) * P + tin + r]);
        }
        if (have) {
            key_codes<BITS>(base, (int64_t)(tin + r) * (D / 8) + (j & 3) * (D / 32) + (j >> 2), x[i][0]);
            value_codes<BITS>(base + pl.v_codes, (int64_t)(tin >> 3) * D + 8 * j, r, x[i][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < kReadBlocks; ++i) {
        const int64_t t = tok8 + 8 * i + r;
        const bool on = t >= f0 && t < f0 + n;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            s16x2(&w)[4] = x[i][kv];
            float y[8];
            uint32_t sb = 0;
            if constexpr (ROT) {
                fwht_pairs(w, j);
                if ((j & 7) == 0) w[0].x -= 64 * off;
                const float s = sc[i][kv] * (D == 128 ? 0.08838834764831845f : 0.125f);
                sb = sign_byte(kv ? a.c.sv : a.c.sk, j);
                s16x2 o[4];
                float so = 0.f;
                if constexpr (D == 128) {
                    // feature f + 64 of the row is I0 - I1 where f is I0 + I1
                    so = lane_xor<8>(s);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = lane_xor_pair<8>(w[e]);
                }
                const float own = (j & 8) ? -s : s;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = (float)(e & 1 ? w[e >> 1].y : w[e >> 1].x);
                    if constexpr (D == 128) y[e] = fmaf(v, own, (float)(e & 1 ? o[e >> 1].y : o[e >> 1].x) * so);
                    else y[e] = v * s;
                }
            } else {
                const float s = sc[i][kv], c = -(float)off * s;          // exact: (u - off) s in one rounding
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fmaf((float)(e & 1 ? w[e >> 1].y : w[e >> 1].x), s, c);
            }
            if (on) {
                const RowsView &dst = kv ? a.v : a.k;
                store8(static_cast<T *>(dst.ptr) + ((int64_t)s0 + (t - f0)) * dst.ts + id.h * dst.hs + 8 * j, y, sb);
            }
        }
    }
}

// ---------------------------------------------------------------- keep
// One workgroup of 256 threads per (sequence, head): the kept tokens' K units,
// V codes and scales are all gathered into LDS, then written to their places.
template <int D, int BITS>
__global__ __launch_bounds__(256) void k_cache_keep(CacheKeepArgs a) {
    const int h = blockIdx.x % a.c.H, b = blockIdx.x / a.c.H, tid = threadIdx.x;
    int s0;
    const int n = min(ragged_rows(a.starts, b, a.total, &s0), kMaxKeep);
    const int base = a.base[b];
    if (n == 0 || base < 0 || base > (a.c.max_pages << a.c.page_shift)) return;
    const int P = 1 << a.c.page_shift;
    const PageLayout pl = page_layout(P, D, BITS);
    constexpr int NU = D / 8;
    __shared__ uint2 ku[kMaxKeep][NU];
    __shared__ uint8_t vc[kMaxKeep][D];
    __shared__ uint16_t sc[kMaxKeep][2 * (D / 64)];
    __shared__ int64_t dst[kMaxKeep];                // pool offset of the target's page block, -1: leave it
    __shared__ int64_t src[kMaxKeep];
    __shared__ int tsrc[kMaxKeep];
    if (tid < n) {
        const int p = a.path[s0 + tid];
        const bool ok = p >= 0 && p < kMaxKeep;
        const int ps = ok ? cache_page(a.c, b, base + p) : -1, pd = cache_page(a.c, b, base + tid);
        tsrc[tid] = base + (ok ? p : 0);
        src[tid] = ps >= 0 && pd >= 0 ? cache_block_offset(a.c, ps, h) : -1;
        dst[tid] = ps >= 0 && pd >= 0 ? cache_block_offset(a.c, pd, h) : -1;
    }
    __syncthreads();
    for (int i = tid; i < n * NU; i += 256) {
        const int r = i / NU, u = i % NU;
        if (src[r] >= 0) ku[r][u] = load_unit<BITS>(a.c.pool + src[r], (int64_t)(tsrc[r] & (P - 1)) * NU + u);
    }
    for (int i = tid; i < n * D; i += 256) {
        const int r = i / D, f = i % D, t = tsrc[r] & (P - 1);
        if (src[r] >= 0)
            vc[r][f] = (uint8_t)unit_code<BITS>(load_unit<BITS>(a.c.pool + src[r] + pl.v_codes, (int64_t)(t >> 3) * D + f),
                                                t & 7);
    }
    for (int i = tid; i < n * 2 * (D / 64); i += 256) {
        const int r = i / (2 * (D / 64)), g = i % (2 * (D / 64));      // K groups, then V groups
        if (src[r] >= 0)
            sc[r][g] = reinterpret_cast<const uint16_t *>(a.c.pool + src[r] + pl.k_scales)[g * P + (tsrc[r] & (P - 1))];
    }
    __syncthreads();
    for (int i = tid; i < n * NU; i += 256) {
        const int r = i / NU, u = i % NU;
        if (dst[r] >= 0) store_unit<BITS>(a.c.pool + dst[r], (int64_t)((base + r) & (P - 1)) * NU + u, ku[r][u]);
    }
    for (int i = tid; i < n * 2 * (D / 64); i += 256) {
        const int r = i / (2 * (D / 64)), g = i % (2 * (D / 64));
        if (dst[r] >= 0)
            reinterpret_cast<uint16_t *>(a.c.pool + dst[r] + pl.k_scales)[g * P + ((base + r) & (P - 1))] = sc[r][g];
    }
    // V: a thread owns feature f of a block of 8 targets
    const int blk0 = base >> 3, nb = ((base + n - 1) >> 3) - blk0 + 1;
    for (int i = tid; i < nb * D; i += 256) {
        const int blk = blk0 + i / D, f = i % D;
        uint2 m = make_uint2(0, 0), w = make_uint2(0, 0);
        int64_t at = -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int r = blk * 8 + e - base;
            if (r < 0 || r >= n || dst[r] < 0) continue;
            at = dst[r];
            const uint32_t c = vc[r][f];
            const uint2 me = member_mask<BITS>(e);
            m.x |= me.x;
            m.y |= me.y;
            if constexpr (BITS == 4) w.x |= c << nibble_of(e);
            else if (e < 4) w.x |= c << (8 * e);
            else w.y |= c << (8 * (e - 4));
        }
        if (at < 0) continue;
        uint8_t *codes = a.c.pool + at + pl.v_codes;
        const int64_t unit = (int64_t)((blk * 8 & (P - 1)) >> 3) * D + f;
        const uint2 o = load_unit<BITS>(codes, unit);
        store_unit<BITS>(codes, unit, make_uint2((o.x & ~m.x) | w.x, (o.y & ~m.y) | w.y));
    }
}

// ---------------------------------------------------------------- launchers
// blocks of 8 tokens that at most n consecutive tokens touch
static int64_t blocks8(int n) { return ((int64_t)n + 6) / 8 + 1; }

template <typename T, int D, int BITS, bool ROT>
static hipError_t rows_launch(const CacheRowsArgs &a, bool read, hipStream_t s) {
    const int64_t b8 = blocks8(a.max_rows), nblk = read ? (b8 + kReadBlocks - 1) / kReadBlocks : b8;
    const int64_t grid = nblk * a.c.H * a.c.batch;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (read) hipLaunchKernelGGL((k_cache_read<T, D, BITS, ROT>), dim3((unsigned)grid), dim3(D), 0, s, a, (int)nblk);
    else hipLaunchKernelGGL((k_cache_append<T, D, BITS, ROT>), dim3((unsigned)grid), dim3(D), 0, s, a, (int)nblk);
    return hipGetLastError();
}
template <typename T, int D, int BITS>
static hipError_t rows_rot(const CacheRowsArgs &a, bool rotate, bool read, hipStream_t s) {
    return rotate ? rows_launch<T, D, BITS, true>(a, read, s) : rows_launch<T, D, BITS, false>(a, read, s);
}
template <typename T>
static hipError_t rows_t(const CacheRowsArgs &a, int d, int bits, bool rotate, bool read, hipStream_t s) {
    if (d == 128) return bits == 4 ? rows_rot<T, 128, 4>(a, rotate, read, s) : rows_rot<T, 128, 8>(a, rotate, read, s);
    return bits == 4 ? rows_rot<T, 64, 4>(a, rotate, read, s) : rows_rot<T, 64, 8>(a, rotate, read, s);
}
hipError_t launch_cache_append(const CacheRowsArgs &a, int d, int bits, int dtype, bool rotate, hipStream_t s) {
    KTimeScope kts("k_cache_append", s);
    return dtype == JOLT_BF16 ? rows_t<uint16_t>(a, d, bits, rotate, false, s)
                              : rows_t<float>(a, d, bits, rotate, false, s);
}
hipError_t launch_cache_read(const CacheRowsArgs &a, int d, int bits, int dtype, bool rotate, hipStream_t s) {
    KTimeScope kts("k_cache_read", s);
    return dtype == JOLT_BF16 ? rows_t<uint16_t>(a, d, bits, rotate, true, s)
                              : rows_t<float>(a, d, bits, rotate, true, s);
}
hipError_t launch_cache_keep(const CacheKeepArgs &a, int d, int bits, hipStream_t s) {
    KTimeScope kts("k_cache_keep", s);
    const int64_t grid = (int64_t)a.c.batch * a.c.H;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    const dim3 g((unsigned)grid), t(256);
    if (d == 128 && bits == 4) hipLaunchKernelGGL((k_cache_keep<128, 4>), g, t, 0, s, a);
    else if (d == 128) hipLaunchKernelGGL((k_cache_keep<128, 8>), g, t, 0, s, a);
    else if (bits == 4) hipLaunchKernelGGL((k_cache_keep<64, 4>), g, t, 0, s, a);
    else hipLaunchKernelGGL((k_cache_keep<64, 8>), g, t, 0, s, a);
    return hipGetLastError();
}

}  // namespace jolt
