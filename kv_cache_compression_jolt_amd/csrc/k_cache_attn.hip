// Attention over the token cache (jolt_cache_attention, jolt_tree_attention).
//
// For a query row q of KV head h, with u the stored codes (unsigned, offset
// c0), sc_g the scale of group g of 64 features and q' the query in the cache's
// domain (rotated: q' = (1/sqrt d) H (s o q)):
//   q . k_t = sum_g sc_g[t] (sum_{f in g} q'_f u_f[t] - c0 sum_{f in g} q'_f)
//   o'_f    = sum_t w_g[t] u_f[t] - c0 sum_t w_g[t],   w_g[t] = p_t sc_g^V[t]
// and o = o' / sum p, rotated back once per row.  So the codes go into the
// matrix cores as they are stored, as integers, exact in bf16; the offset is
// the accumulator's initial value for the scores and one extra product with a
// row of ones for the values; scales are applied to scores and weights in fp32.
// A 4-bit code becomes bf16 by or-ing it under the exponent of 128 (value
// 128 + u, c0 = 136), two codes per and-or.
//
// Products are S^T = K Q^T and O^T = V^T P^T (16x16x32): a lane then holds one
// query column and 8 tokens' scores, in exactly the order that the second
// product takes its P^T operand in, so weights never leave registers.  Softmax
// runs in one pass with a running maximum per column, which is raised, and the
// sums rescaled, only when a score passes it by 2^8.
//
// Roundings: K and V codes are exact; a rotated query is held in two bf16 parts
// (one part alone would err by 2^-9 of every feature, and the scores with it); a
// weight times its value scale is rounded to bf16, because the product takes it so:
// 2^-9 of each summand, as in any attention on 16-bit weights.
//
// Bound by the reads of the cache for one token a sequence, and at long ranges by
// how many are in flight: two blocks of 32 tokens a wave, two workgroups a CU.
// d = 128, 8 heads, 32 query heads: 16 x 8192 tokens of 8 bits 51 us with the join
// (3.2 TB/s; a large copy 5.1), 65535 tokens of 4 bits 26.6 us (2.7 TB/s).  At 32
// and more columns the vector work that turns codes into bf16 is done again for
// every 16 columns and bounds it: 61 us for 48 columns over 16 x 4096 tokens.
#include <algorithm>

#include "cache.h"
#include "cache_attn_dev.h"
#include "jolt_internal.h"
#include "ktimer.h"

namespace jolt {

namespace {

constexpr int kCols = 16;                 // query columns of a tile
constexpr int kWaves = 4;

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

template <int BITS> constexpr float code_offset() { return BITS == 4 ? 136.f : 128.f; }

__device__ __forceinline__ float scale_of(const uint32_t *w, int e) {
    return __uint_as_float((e & 1) ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16));
}

// One wave's share of a 32-token block as it lies in memory
template <int D, int BITS>
struct BlockRegs {
    static constexpr int kU = BITS / 4;                 // dwords of a unit
    static constexpr int kK = D / 32 * kU;              // K dwords of a lane and subtile
    static constexpr int kV = D / 16 * kU;              // V dwords of a lane
    uint32_t k[2][kK], v[kV], ks[D / 64][4], vs[D / 64][4];

    // tokens t0 .. t0 + 31, inside one page; lane (m, g): K chunk g of token
    // rows 8 (m/4) + 4 u + m%4, V units of tokens 8 g .. 8 g + 7, and those
    // tokens' scales
    __device__ __forceinline__ void load(const uint8_t *blk, const PageLayout &pl, int P, int tin, int m, int g) {
        constexpr int rowb = D * BITS / 8;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            load_dwords<kK>(blk + (tin + 8 * (m >> 2) + 4 * u + (m & 3)) * rowb + g * (rowb / 4), k[u]);
        const uint8_t *vp = blk + pl.v_codes + ((tin >> 3) + g) * (D * BITS);
#pragma unroll
        for (int i = 0; i < kV; i += 4) {
            uint32_t t[4];
            load_dwords<4>(vp + i * 64 + m * 16, t);     // 16 lanes x 16 bytes per step
#pragma unroll
            for (int x = 0; x < 4; ++x) v[i + x] = t[x];
        }
#pragma unroll
        for (int q = 0; q < D / 64; ++q) {
            load_dwords<4>(blk + pl.k_scales + (q * P + tin + 8 * g) * 2, ks[q]);
            load_dwords<4>(blk + pl.v_scales + (q * P + tin + 8 * g) * 2, vs[q]);
        }
    }
};
// the feature that row m of value tile i stands for (the order of the 16-byte loads)
template <int BITS>
__device__ __forceinline__ constexpr int value_feature(int i, int m) {
    constexpr int per = 16 / BITS;                      // units (features) of a 16-byte load
    return (i / per) * (16 * per) + m * per + i % per;
}

}  // namespace

// ---------------------------------------------------------------- attention
// One workgroup of 4 waves per (token range, KV head, tile of 16 query columns,
// sequence); column c of a sequence's KV head is query row c / G, head h G +
// c % G.  The waves take the range's 32-token blocks in turn (each block's
// fragments go from memory to registers, the next block's while this one is
// computed) and join their sums through LDS at the end.  No tile goes through LDS:
// with 16 columns each fragment is used by one wave once.
template <int D, int BITS, bool ROT>
__global__ __launch_bounds__(64 * kWaves, 2) void k_cache_attn(CacheAttnArgs a, int ctiles) {
    constexpr int NK = D / 32, NV = D / 16, NG = D / 64, KU = BITS / 4;
    const AttnTile id = attn_tile(a, ctiles);
    if (!id.valid) return;
    const int b = id.b, h = id.h, ct = id.ct, split = id.split;
    int s0;
    const int nall = ragged_rows(a.starts, b, a.total, &s0), n = min(nall, a.max_q);
    if (ct * kCols >= n * a.G) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, m = lane & 15, g = lane >> 4;
    const int len = cache_len(a.c, b), base = a.c.lens[b] - nall;
    const int prefix = a.prefix ? a.prefix[b] : 0;

    __shared__ __align__(16) float sm[kWaves * kCols * (D + 4)];
    __shared__ float sml[2][kWaves][kCols];

    // ---- what the columns see
    const int c = ct * kCols + m, ncol = n * a.G;
    const bool cv = c < ncol;
    const Column col(a, s0, n, base, len, prefix, h, c, cv);
    Reach reach(col, cv);
    reach.join<16>();
    reach.clip(a, len, prefix);
    reach.uniform();
    const int lo_any = reach.lo_any, hi_any = reach.hi_any, lo_all = reach.lo_all, hi_all = reach.hi_all;
    const int begin = reach.begin(prefix);

    // ---- this workgroup's blocks
    const int blk0 = begin >> 5, nblk = hi_any > begin ? ((hi_any + 31) >> 5) - blk0 : 0;
    const int per = max((nblk + a.splits - 1) / a.splits, a.least >> 5);
    const int bs = blk0 + split * per, be = min(bs + per, blk0 + nblk);

    const int P = 1 << a.c.page_shift;
    const PageLayout pl = page_layout(P, D, BITS);
    // ---- this wave's blocks: bs + wave, then every kWaves-th.  The page numbers of
    // its next 64 blocks sit in one register (lane i: block seen + i kWaves), and
    // the first block's loads start before the queries are prepared.
    int seen = bs + wave, pages = -1;
    auto load_pages = [&]() {
        const int blk = seen + lane * kWaves, t0 = blk << 5;
        // blocks between a prefix and the window hold nothing visible
        pages = blk < be && (t0 < prefix || t0 + 32 > lo_any) ? cache_page(a.c, b, t0) : -1;
    };
    auto page_of = [&](int blk) -> int {
        if (blk >= be) return -1;
        if (blk - seen >= 64 * kWaves) {
            seen = blk;
            load_pages();
        }
        return __builtin_amdgcn_readlane(pages, (blk - seen) / kWaves);
    };
    BlockRegs<D, BITS> even, odd;
    auto load = [&](BlockRegs<D, BITS> &r, int blk, int page) {
        if (page >= 0) r.load(a.c.pool + cache_block_offset(a.c, page, h), pl, P, (blk << 5) & (P - 1), m, g);
    };
    load_pages();
    int page = page_of(bs + wave);
    load(even, bs + wave, page);

    // ---- the queries in the cache's domain, one row per D / 8 lanes, through LDS
    {
        const int r = tid / (D / 8), j = tid % (D / 8);
        if (D == 128 || tid < 128) {
            const int c = ct * kCols + r;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
            if (c < n * a.G) {
                const int i = c / a.G, hd = h * a.G + c % a.G;
                const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q.ptr) +
                                                                 (int64_t)(s0 + i) * a.q.ts + hd * a.q.hs + 8 * j);
                const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = scale_of(q, e);
            }
            if constexpr (ROT) {
                const uint32_t sb = sign_byte(a.c.sk, j);
                const float isd = D == 128 ? 0.08838834764831845f : 0.125f;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = flip(x[e], (sb >> e) & 1);
                fwht_row<D>(x, j);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= isd;
            }
            float4 *p = reinterpret_cast<float4 *>(sm + r * (D + 4) + 8 * j);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
    __syncthreads();
    // fragments: column m, features 32 k + 8 g + e; hi and (rotated) lo parts;
    // cinit: minus the offset times the column's sum over each group
    constexpr int NP = ROT ? 2 : 1;
    bf16x8 qf[NP][NK];
    float cinit[NG];
#pragma unroll
    for (int q = 0; q < NG; ++q) cinit[q] = 0.f;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
        const float *p = sm + m * (D + 4) + 32 * k + 8 * g;
        float sum = 0.f;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = p[2 * i], x1 = p[2 * i + 1];
            hi[i] = bf16_pair(x0, x1);
            const float h0 = __uint_as_float(hi[i] << 16), h1 = __uint_as_float(hi[i] & 0xFFFF0000u);
            sum += h0 + h1;
            if constexpr (ROT) {
                lo[i] = bf16_pair(x0 - h0, x1 - h1);
                sum += __uint_as_float(lo[i] << 16) + __uint_as_float(lo[i] & 0xFFFF0000u);
            }
        }
        qf[0][k] = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        if constexpr (ROT) qf[NP - 1][k] = __builtin_bit_cast(bf16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        cinit[k / 2] += sum;
    }
#pragma unroll
    for (int q = 0; q < NG; ++q) {
        cinit[q] += __shfl_xor(cinit[q], 16);
        cinit[q] += __shfl_xor(cinit[q], 32);
        cinit[q] *= -code_offset<BITS>();
    }
    __syncthreads();                                    // sm is reused by the join

    f32x4 acc[NV], corr[NG];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < NG; ++q) corr[q] = f32x4{0.f, 0.f, 0.f, 0.f};
    float mrun = neg_inf(), lrun = 0.f;
    const float mul = a.scale * kLog2e, cap_mul = a.cap > 0.f ? a.scale / a.cap * (2.f * kLog2e) : 0.f;
    const bf16x8 ones = __builtin_bit_cast(bf16x8, make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u));

    auto work = [&](const BlockRegs<D, BITS> &use, int blk) {
        const int t0 = blk << 5;
        // scores: lane (column m) has tokens t0 + 8 g + e
        float s[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int q = 0; q < NG; ++q) {
                f32x4 x = {cinit[q], cinit[q], cinit[q], cinit[q]};
#pragma unroll
                for (int k = 2 * q; k < 2 * q + 2; ++k) {
                    const bf16x8 kf = unit_bf16<BITS>(&use.k[u][k * KU]);
#pragma unroll
                    for (int p = 0; p < NP; ++p) x = mfma16(kf, qf[p][k], x);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float ks = scale_of(use.ks[q], 4 * u + i);
                    s[4 * u + i] = q == 0 ? x[i] * ks : fmaf(x[i], ks, s[4 * u + i]);
                }
            }
        }
        if (a.cap > 0.f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {           // tanh |y| = (1 - x) / (1 + x), x = exp(-2 |y|)
                const float x = __builtin_amdgcn_exp2f(-fabsf(s[e] * cap_mul));
                s[e] = copysignf((1.f - x) * __builtin_amdgcn_rcpf(1.f + x), s[e]) * (a.cap * kLog2e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] *= mul;
        }
        const bool full = t0 >= lo_all && t0 + 32 <= hi_all;
        if (a.slopes) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] -= col.slope * col.distance(a, t0 + 8 * g + e, s0, n, base);
        }
        uint32_t vis = 0xFFu;
        if (!full) {
            vis = col.sees8(a.tree != nullptr, base, t0 + 8 * g);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = (vis >> e) & 1 ? s[e] : neg_inf();
        }
        float mx = s[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[e]);
        if (__any(mx > mrun + 8.f)) {
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            mx = fmaxf(mx, mrun);
            const float alpha = mx == mrun ? 1.f : __builtin_amdgcn_exp2f(mrun - mx);
            mrun = mx;
            lrun *= alpha;
#pragma unroll
            for (int i = 0; i < NV; ++i) acc[i] *= alpha;
#pragma unroll
            for (int q = 0; q < NG; ++q) corr[q] *= alpha;
        }
        const float mu = mrun == neg_inf() ? 0.f : mrun;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(s[e] - mu);
            lrun += p[e];
        }
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            uint32_t wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float w0 = p[2 * i] * scale_of(use.vs[q], 2 * i), w1 = p[2 * i + 1] * scale_of(use.vs[q], 2 * i + 1);
                if (!full) {                        // a masked token's scale may be anything
                    w0 = (vis >> (2 * i)) & 1 ? w0 : 0.f;
                    w1 = (vis >> (2 * i + 1)) & 1 ? w1 : 0.f;
                }
                wv[i] = bf16_pair(w0, w1);
            }
            const bf16x8 wf = __builtin_bit_cast(bf16x8, make_uint4(wv[0], wv[1], wv[2], wv[3]));
            corr[q] = mfma16(ones, wf, corr[q]);
#pragma unroll
            for (int i = q * (NV / NG); i < (q + 1) * (NV / NG); ++i)
                acc[i] = mfma16(unit_bf16<BITS>(&use.v[i * KU]), wf, acc[i]);
        }
    };
    for (int blk = bs + wave; blk < be; blk += 2 * kWaves) {
        int next = page_of(blk + kWaves);
        load(odd, blk + kWaves, next);
        if (page >= 0) work(even, blk);
        page = next;
        next = page_of(blk + 2 * kWaves);
        load(even, blk + 2 * kWaves, next);
        if (page >= 0) work(odd, blk + kWaves);
        page = next;
    }

    // ---- join the waves
    lrun += __shfl_xor(lrun, 16);
    lrun += __shfl_xor(lrun, 32);
    mrun = nan_outweighs(mrun, lrun);
    if (g == 0) {
        sml[0][wave][m] = mrun;
        sml[1][wave][m] = lrun;
    }
    __syncthreads();
    {
        float mx = sml[0][0][m];
#pragma unroll
        for (int x = 1; x < kWaves; ++x) mx = fmaxf(mx, sml[0][x][m]);
        const float f = mrun == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(mrun - mx);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float o = acc[i][x] - code_offset<BITS>() * corr[i / (NV / NG)][x];
                sm[(wave * kCols + m) * (D + 4) + value_feature<BITS>(i, 4 * g + x)] = mrun == neg_inf() ? 0.f : o * f;
            }
    }
    __syncthreads();
    const int r = tid / (D / 8), j = tid % (D / 8), cr = ct * kCols + r;
    if (D == 64 && r >= kCols) return;
    float mx = sml[0][0][r], l = 0.f;
#pragma unroll
    for (int x = 1; x < kWaves; ++x) mx = fmaxf(mx, sml[0][x][r]);
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
        if (sml[0][x][r] != neg_inf()) l += sml[1][x][r] * __builtin_amdgcn_exp2f(sml[0][x][r] - mx);
        const float4 *p = reinterpret_cast<const float4 *>(sm + (x * kCols + r) * (D + 4) + 8 * j);
        const float4 u = p[0], v = p[1];
        o[0] += u.x; o[1] += u.y; o[2] += u.z; o[3] += u.w;
        o[4] += v.x; o[5] += v.y; o[6] += v.z; o[7] += v.w;
    }
    const int64_t row = s0 + cr / a.G;
    const int head = h * a.G + cr % a.G;
    if (a.splits == 1) {
        finish_row<D, ROT>(a, row, head, j, o, mx, l, cr < ncol);
    } else if (cr < ncol) {
        const int64_t rows = (int64_t)a.total * a.hq, at = split * rows + row * a.hq + head;
        if (j == 0) {
            a.ws_ml[2 * at] = mx;
            a.ws_ml[2 * at + 1] = l;
        }
        if (mx != neg_inf()) {
            float4 *p = reinterpret_cast<float4 *>(a.ws_part + at * D + 8 * j);
            p[0] = make_float4(o[0], o[1], o[2], o[3]);
            p[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
    }
}

// ---------------------------------------------------------------- joining token ranges
// o = sum_s 2^(m_s - m) o_s, l likewise, over the ranges s of a row; a range in
// which the row saw nothing (m_s = -inf) has no sums in the workspace.  Rows are
// addressed through the sequences, so rows that no sequence has stay as they are.

// Up to kFew ranges: D / 8 lanes take a row's ranges one after the other.  Bound by
// the launch and a chain of loads: 3.4 us for a decode step of 16 sequences, 5.8
// for the 48 rows each of 16 trees.
constexpr int kFew = 16;
template <int D, bool ROT>
__global__ __launch_bounds__(256) void k_cache_attn_join(CacheAttnArgs a, int nblk) {
    constexpr int NGRP = 2048 / D;
    const int b = blockIdx.x / nblk, blk = blockIdx.x % nblk;
    int s0;
    const int n = min(ragged_rows(a.starts, b, a.total, &s0), a.max_q);
    const int grp = threadIdx.x / (D / 8), j = threadIdx.x % (D / 8), r = blk * NGRP + grp;
    if (blk * NGRP >= n * a.hq) return;
    const bool on = r < n * a.hq;
    const int row = s0 + (on ? r / a.hq : 0), head = on ? r % a.hq : 0;
    const int64_t rows = (int64_t)a.total * a.hq, at = (int64_t)row * a.hq + head;
    float m = neg_inf(), l = 0.f, o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float2 ml = *reinterpret_cast<const float2 *>(a.ws_ml + 2 * (s * rows + at));
        const float4 *p = reinterpret_cast<const float4 *>(a.ws_part + (s * rows + at) * D + 8 * j);
        const float4 x = p[0], y = p[1];
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        const bool none = ml.x == neg_inf();
        const float mn = fmaxf(m, ml.x);
        const float f0 = m == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(m - mn), f1 = none ? 0.f : __builtin_amdgcn_exp2f(ml.x - mn);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(o[e], f0, none ? 0.f : v[e] * f1);
        l = fmaf(l, f0, none ? 0.f : ml.y * f1);
        m = mn;
    }
    finish_row<D, ROT>(a, row, head, j, o, m, l, on);
}

// More: one workgroup of 256 threads per row.  Every thread first takes one
// range's m and l, so that all weights are known after one read; then 2048 / D
// groups of D / 8 lanes sum the ranges in turn and are added through LDS.  64
// ranges of a 64 k cache: 4.1 us.
constexpr int kMaxSplits = 256;
template <int D, bool ROT>
__global__ __launch_bounds__(256) void k_cache_attn_join_many(CacheAttnArgs a) {
    constexpr int NGRP = 2048 / D;
    const int b = blockIdx.x / (a.max_q * a.hq), r = blockIdx.x % (a.max_q * a.hq);
    int s0;
    const int n = min(ragged_rows(a.starts, b, a.total, &s0), a.max_q);
    if (r >= n * a.hq) return;
    const int row = s0 + r / a.hq, head = r % a.hq, tid = threadIdx.x;
    const int64_t rows = (int64_t)a.total * a.hq, at = (int64_t)row * a.hq + head;
    __shared__ float so[NGRP][D + 4], sw[kMaxSplits], red[2][4];
    const float2 ml = tid < a.splits ? *reinterpret_cast<const float2 *>(a.ws_ml + 2 * (tid * rows + at))
                                     : make_float2(neg_inf(), 0.f);
    const float mw = wave_max(ml.x);
    if ((tid & 63) == 0) red[0][tid >> 6] = mw;
    __syncthreads();
    const float m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float w = ml.x == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(ml.x - m);
    sw[tid] = w;
    const float lw = wave_sum(w == 0.f ? 0.f : w * ml.y);
    if ((tid & 63) == 0) red[1][tid >> 6] = lw;
    __syncthreads();
    const float l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    const int grp = tid / (D / 8), j = tid % (D / 8);
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int s = grp; s < a.splits; s += NGRP) {
        const float4 *p = reinterpret_cast<const float4 *>(a.ws_part + (s * rows + at) * D + 8 * j);
        const float4 x = p[0], y = p[1];
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}, f = sw[s];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += f == 0.f ? 0.f : v[e] * f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) so[grp][8 * j + e] = o[e];
    __syncthreads();
    if (tid >= 64) return;                              // one wave (whole, for the lane exchanges) finishes the row
    const int jj = tid % (D / 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
    for (int x = 0; x < NGRP; ++x)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += so[x][8 * jj + e];
    finish_row<D, ROT>(a, row, head, jj, o, m, l, tid < D / 8);
}

// ---------------------------------------------------------------- launchers
template <int D, int BITS, bool ROT>
static hipError_t attn_launch(const CacheAttnArgs &a, hipStream_t s) {
    const int ctiles = (int)(((int64_t)a.max_q * a.G + kCols - 1) / kCols);
    const int64_t grid = attn_grid((int64_t)a.c.batch * a.c.H, (int64_t)a.splits * ctiles);
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    KTimeScope kts("k_cache_attn", s);
    hipLaunchKernelGGL((k_cache_attn<D, BITS, ROT>), dim3((unsigned)grid), dim3(64 * kWaves), 0, s, a, ctiles);
    return hipGetLastError();
}
template <int D>
static hipError_t attn_d(const CacheAttnArgs &a, bool wide, int bits, bool rotate, hipStream_t s) {
    hipError_t e;
    if (wide) e = launch_cache_attn_wide(a, D, bits, rotate, s);
    else if (bits == 4) e = rotate ? attn_launch<D, 4, true>(a, s) : attn_launch<D, 4, false>(a, s);
    else e = rotate ? attn_launch<D, 8, true>(a, s) : attn_launch<D, 8, false>(a, s);
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t rows = (int64_t)a.max_q * a.hq, many = rows * a.c.batch, nblk = (rows * D + 2047) / 2048;
    if (many > 0x7FFFFFFF) return hipErrorInvalidValue;
    KTimeScope kts("k_cache_attn_join", s);
    const dim3 gf((unsigned)(nblk * a.c.batch)), gm((unsigned)many), t(256);
    if (a.splits <= kFew) {
        if (rotate) hipLaunchKernelGGL((k_cache_attn_join<D, true>), gf, t, 0, s, a, (int)nblk);
        else hipLaunchKernelGGL((k_cache_attn_join<D, false>), gf, t, 0, s, a, (int)nblk);
    } else {
        if (rotate) hipLaunchKernelGGL((k_cache_attn_join_many<D, true>), gm, t, 0, s, a);
        else hipLaunchKernelGGL((k_cache_attn_join_many<D, false>), gm, t, 0, s, a);
    }
    return hipGetLastError();
}
hipError_t launch_cache_attention(const CacheAttnArgs &a, bool wide, int d, int bits, bool rotate, hipStream_t s) {
    return d == 128 ? attn_d<128>(a, wide, bits, rotate, s) : attn_d<64>(a, wide, bits, rotate, s);
}

}  // namespace jolt
