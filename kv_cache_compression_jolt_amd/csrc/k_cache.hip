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
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// store 8 values, with the signs changed of those whose bit (15 or 31 of the
// pair's word) is set
template <typename T> __device__ __forceinline__ void store8_signed(T *p, const float (&x)[8], const uint32_t *neg);
template <> __device__ __forceinline__ void store8_signed<uint16_t>(uint16_t *p, const float (&x)[8], const uint32_t *neg) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(bf16_pair(x[0], x[1]) ^ neg[0], bf16_pair(x[2], x[3]) ^ neg[1],
                                               bf16_pair(x[4], x[5]) ^ neg[2], bf16_pair(x[6], x[7]) ^ neg[3]);
}
template <> __device__ __forceinline__ void store8_signed<float>(float *p, const float (&x)[8], const uint32_t *neg) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        y[e] = __uint_as_float(__float_as_uint(x[e]) ^ ((e & 1) ? neg[e >> 1] & 0x80000000u : neg[e >> 1] << 16));
    reinterpret_cast<float4 *>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}
// store 8 values of a row that the neighbouring lanes complete in the same
// instruction: whole lines of bf16 go past the caches (39 -> 34 us for the read
// of 12k tokens of 8 heads; the rotated reader's 64-byte pieces lose by it, 176
// -> 199 us for 16 x 8192 tokens)
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&x)[8]);
template <> __device__ __forceinline__ void store8<uint16_t>(uint16_t *p, const float (&x)[8]) {
    const u32x4 v = {bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}
template <> __device__ __forceinline__ void store8<float>(float *p, const float (&x)[8]) {
    constexpr uint32_t none[4] = {0, 0, 0, 0};
    store8_signed(p, x, none);
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
//
// Bound by memory for many rows (each is read once, its codes written once): a
// workgroup's 8 tokens make whole V units, so nothing is written twice, and the
// heads of a token run side by side where the rows lie that way.  Prompts of up to
// 4097 tokens, 5 sequences, 8 heads, d = 128, 8 bits: 18-21 us, with the read of
// the same rows 34 us (4.5 TB/s over both; a large copy reaches 5.1).  For a
// decode step of 64 rows the launch and one chain of dependent loads are left: 6 us.
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
    const int tid = threadIdx.x, j = tid % (D / 8), r = tid / (D / 8), t = tok8 + r;
    const bool on = t >= from && t <= last;
    const int64_t row = (int64_t)s0 + (t - t0);
    __shared__ __align__(16) uint8_t vc[8][D];
    // both rows, and the V units that the block keeps other tokens in, are under
    // way before any is used
    float in[2][8];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const RowsView &src = kv ? a.v : a.k;
#pragma unroll
        for (int e = 0; e < 8; ++e) in[kv][e] = 0.f;
        if (on) load8(static_cast<const T *>(src.ptr) + row * src.ts + id.h * src.hs + 8 * j, in[kv]);
    }
    const int page = cache_page(a.c, id.b, tok8);
    if (page < 0) return;
    uint8_t *base = a.c.pool + cache_block_offset(a.c, page, id.h);
    const int P = 1 << a.c.page_shift, tin = tok8 & (P - 1);
    const PageLayout pl = page_layout(P, D, BITS);
    const int64_t unit = (int64_t)(tin >> 3) * D + tid;
    const bool part = tok8 < from || tok8 + 7 > last;
    const uint2 old = part ? load_unit<BITS>(base + pl.v_codes, unit) : make_uint2(0, 0);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float(&x)[8] = in[kv];
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
    if (part) {
        uint2 m = make_uint2(0, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (tok8 + e >= from && tok8 + e <= last) {
                const uint2 me = member_mask<BITS>(e);
                m.x |= me.x;
                m.y |= me.y;
            }
        w.x = (w.x & m.x) | (old.x & ~m.x);
        w.y = (w.y & m.y) | (old.y & ~m.y);
    }
    store_unit<BITS>(base + pl.v_codes, unit, w);
}

// ---------------------------------------------------------------- read
// Rows stored as they are: a thread (row r, lane j of D / 8) rebuilds features
// 8 j .. 8 j + 7 of one token of a block of 8, and does so for kReadBlocks blocks
// at once, so that their loads are in flight together.  Bound by the stores: 15-16
// us for the prompts of up to 4097 tokens above; 4.2 us for 3 x 701 rows in fp32.
constexpr int kReadBlocks = 2;

// member e of the units of 8 consecutive features, one a dword
template <int BITS>
__device__ __forceinline__ void value_words(const uint8_t *codes, int64_t unit, int e, uint32_t (&w)[8]) {
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
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] >>= sh;
}

template <typename T, int D, int BITS>
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
    constexpr float off = (float)(1 << (BITS - 1));
    float x[kReadBlocks][2][8], sc[kReadBlocks][2];
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
            for (int e = 0; e < 8; ++e) x[i][kv][e] = 0.f;
            if (have)
                sc[i][kv] = bf16_to_f32(reinterpret_cast<const uint16_t *>(base + (kv ? pl.v_scales : pl.k_scales))[(j >> 3) * P + tin + r]);
        }
        if (have) {
            const uint2 k = load_unit<BITS>(base, (int64_t)(tin + r) * (D / 8) + (j & 3) * (D / 32) + (j >> 2));
            uint32_t v[8];
            value_words<BITS>(base + pl.v_codes, (int64_t)(tin >> 3) * D + 8 * j, r, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[i][0][e] = (float)unit_code<BITS>(k, e);
                x[i][1][e] = (float)(v[e] & (BITS == 4 ? 15u : 255u));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kReadBlocks; ++i) {
        const int64_t t = tok8 + 8 * i + r;
        if (t < f0 || t >= f0 + n) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const float s = sc[i][kv], c = -off * s;         // exact: (u - off) s in one rounding
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(x[i][kv][e], s, c);
            const RowsView &dst = kv ? a.v : a.k;
            store8(static_cast<T *>(dst.ptr) + ((int64_t)s0 + (t - f0)) * dst.ts + id.h * dst.hs + 8 * j, y);
        }
    }
}

// Rotated rows: H is symmetric and its own inverse up to d, and the transform of
// a group of 64 integer codes is a matrix product with the +-1 matrix H64, exact
// in bf16 operands and fp32 sums (at most 64 * 255).  One wave takes 64 tokens of
// a head, 16 at a time: products 16x16x32 with A = H64 (rows = features) and B =
// the codes (columns = tokens), the offset of the codes in the initial value of
// feature 0, the only one it reaches.  Rows of A are ordered so that a lane (token
// m, part g) ends with features 8 g .. 8 g + 7 and 32 on from them of each group,
// and four lanes store 64 bytes side by side.  Then
//   y_f = isd (s0 I0 + s1 I1),  y_(f+64) = isd (s0 I0 - s1 I1)   (d = 128)
// with the scales times isd: four roundings.  Bound by memory: 16 tails of 8192
// tokens of 8 heads, 4 bits, take 172-181 us (3.8 TB/s) where their 680 MB take 132
// at the rate of a large copy.  On the vector unit the butterflies cost five times
// the instructions and bounded the kernel (202 us).
template <typename T, int D, int BITS>
__global__ __launch_bounds__(64, 3) void k_cache_read_rot(CacheRowsArgs a, int nblk) {
    constexpr int NG = D / 64, kTok = 64;
    const BlockId id = block_id(a, nblk);
    int s0;
    const int n = min(ragged_rows(a.starts, id.b, a.total, &s0), a.max_rows);
    if (n == 0) return;
    const int64_t f0 = a.first ? a.first[id.b] : 0;
    const int64_t tok = (f0 >> 4) * 16 + (int64_t)id.blk * kTok;
    if (tok >= f0 + n) return;
    const int len = cache_len(a.c, id.b);
    const int lane = threadIdx.x, m = lane & 15, g = lane >> 4;
    const int P = 1 << a.c.page_shift;
    const PageLayout pl = page_layout(P, D, BITS);

    // H64 fragments: row m of tile t is feature f = 32 (t / 2) + 8 (m / 4) + 4 (t % 2) +
    // m % 4; the lane holds columns 32 k + 8 g + e: the signs over e from f's low bits, the rest for all
    bf16x8 hf[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const uint32_t f = 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3);
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p = __popc(f & (2 * i)) & 1;      // element 2 i; 2 i + 1 has f's lowest bit on top
            r[i] = 0x3F803F80u ^ (p << 15) ^ ((p ^ (f & 1)) << 31);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t all = (__popc((f >> 3) & (4 * k + g)) & 1) ? 0x80008000u : 0u;
            hf[t][k] = __builtin_bit_cast(bf16x8, make_uint4(r[0] ^ all, r[1] ^ all, r[2] ^ all, r[3] ^ all));
        }
    }
    // all of the 64 tokens' codes and scales are under way before the first is used;
    // V's go through LDS, from where a lane takes its token's member of 8 units
    constexpr int kBlk = kTok / 16, KU = BITS / 4, KN = D / 32 * KU, VN = D * BITS / 128;
    __shared__ __align__(16) uint32_t vlds[kBlk][VN * 64];
    uint32_t kw[kBlk][KN], vw[kBlk][VN];
    uint16_t sraw[kBlk][2][NG];
#pragma unroll
    for (int blk = 0; blk < kBlk; ++blk) {
        const int64_t t16 = tok + 16 * blk;
        const int page = t16 >= 0 && t16 < len && t16 < f0 + n ? cache_page(a.c, id.b, (int)t16) : -1;
#pragma unroll
        for (int i = 0; i < KN; ++i) kw[blk][i] = 0;
#pragma unroll
        for (int i = 0; i < VN; ++i) vw[blk][i] = 0;
#pragma unroll
        for (int q = 0; q < NG; ++q) sraw[blk][0][q] = sraw[blk][1][q] = 0;
        if (page >= 0) {
            const uint8_t *base = a.c.pool + cache_block_offset(a.c, page, id.h);
            const int tin = (int)(t16 & (P - 1));
            load_dwords<KN>(base + (tin + m) * (D * BITS / 8) + g * (KN * 4), kw[blk]);
            load_dwords<VN>(base + pl.v_codes + (tin >> 3) * (D * BITS) + lane * (VN * 4), vw[blk]);
            if (t16 + m < len)
#pragma unroll
                for (int q = 0; q < NG; ++q) {
                    sraw[blk][0][q] = reinterpret_cast<const uint16_t *>(base + pl.k_scales)[q * P + tin + m];
                    sraw[blk][1][q] = reinterpret_cast<const uint16_t *>(base + pl.v_scales)[q * P + tin + m];
                }
        }
    }
#pragma unroll
    for (int blk = 0; blk < kBlk; ++blk)
#pragma unroll
        for (int i = 0; i < VN; ++i) vlds[blk][lane * VN + i] = vw[blk][i];
    __syncthreads();
    const float isd = D == 128 ? 0.08838834764831845f : 0.125f;
    const float start = g == 0 ? -64.f * (BITS == 4 ? 136.f : 128.f) : 0.f;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        // this lane's output signs, two features to a word, at bits 15 and 31
        uint32_t neg[NG][8];
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            const uint32_t(&sb)[4] = kv ? a.c.sv : a.c.sk;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w = sb[2 * q + (i >> 2)] >> (8 * g + 2 * (i & 3));
                neg[q][i] = ((w & 1u) << 15) | ((w & 2u) << 30);
            }
        }
        const RowsView &dst = kv ? a.v : a.k;
#pragma unroll
        for (int blk = 0; blk < kBlk; ++blk) {
            const int64_t t = tok + 16 * blk + m;
            if (tok + 16 * blk >= f0 + n) break;
            float sc[NG];
            bf16x8 cf[D / 32];
#pragma unroll
            for (int q = 0; q < NG; ++q) sc[q] = bf16_to_f32(sraw[blk][kv][q]);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                if (kv == 0) cf[k] = unit_bf16<BITS>(&kw[blk][k * KU]);
                else {
                    uint32_t w[8], r[4];
                    value_words<BITS>(reinterpret_cast<const uint8_t *>(vlds[blk]), (m >> 3) * D + 32 * k + 8 * g, m & 7, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (BITS == 4)
                            r[i] = (__builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x0C040C00u) & 0x000F000Fu) | 0x43004300u;
                        else
                            r[i] = __builtin_amdgcn_perm(__float_as_uint((float)(w[2 * i + 1] & 255u)),
                                                         __float_as_uint((float)(w[2 * i] & 255u)), 0x07060302u);
                    }
                    cf[k] = __builtin_bit_cast(bf16x8, make_uint4(r[0], r[1], r[2], r[3]));
                }
            }
            f32x4 x[NG][4];
#pragma unroll
            for (int q = 0; q < NG; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[q][i] = f32x4{i == 0 ? start : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        x[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hf[i][k], cf[2 * q + k], x[q][i], 0, 0, 0);
                }
            if (t < f0 || t >= f0 + n) continue;
            T *row = static_cast<T *>(dst.ptr) + ((int64_t)s0 + (t - f0)) * dst.ts + id.h * dst.hs + 8 * g;
            const float sa = sc[0] * isd, sb = NG == 2 ? sc[NG - 1] * isd : 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float lo[8], hi[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = 2 * half + (e >> 2), y = e & 3;
                    lo[e] = x[0][i][y] * sa;
                    if constexpr (NG == 2) {
                        hi[e] = fmaf(x[NG - 1][i][y], -sb, lo[e]);
                        lo[e] = fmaf(x[NG - 1][i][y], sb, lo[e]);
                    }
                }
                store8_signed(row + 32 * half, lo, &neg[0][4 * half]);
                if constexpr (NG == 2) store8_signed(row + 64 + 32 * half, hi, &neg[NG - 1][4 * half]);
            }
        }
    }
}

// ---------------------------------------------------------------- keep
// One workgroup of 256 threads per (sequence, head): the kept tokens' K units,
// V codes and scales are all gathered into LDS, then written to their places, so
// that no token is overwritten before it is read.  A few hundred bytes a token:
// bound by the launch and three dependent loads (starts, path, table, then codes),
// 4.6 us for 16 sequences and for one.
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
// aligned blocks of `size` tokens that at most n consecutive tokens touch
static int64_t blocks_of(int size, int n) { return ((int64_t)n + size - 2) / size + 1; }

template <typename T, int D, int BITS, bool ROT>
static hipError_t rows_launch(const CacheRowsArgs &a, bool read, hipStream_t s) {
    // a rotated read's blocks of 64 tokens begin at a multiple of 16
    const int64_t nblk = !read ? blocks_of(8, a.max_rows)
                               : (ROT ? (16 * blocks_of(16, a.max_rows) + 63) / 64
                                      : (blocks_of(8, a.max_rows) + kReadBlocks - 1) / kReadBlocks);
    const int64_t grid = nblk * a.c.H * a.c.batch;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    const dim3 g((unsigned)grid);
    if (!read) hipLaunchKernelGGL((k_cache_append<T, D, BITS, ROT>), g, dim3(D), 0, s, a, (int)nblk);
    else if constexpr (ROT) hipLaunchKernelGGL((k_cache_read_rot<T, D, BITS>), g, dim3(64), 0, s, a, (int)nblk);
    else hipLaunchKernelGGL((k_cache_read<T, D, BITS>), g, dim3(D), 0, s, a, (int)nblk);
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
