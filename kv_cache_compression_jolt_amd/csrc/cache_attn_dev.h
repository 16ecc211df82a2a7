// Device code shared by the token cache's attention kernels: which tokens a
// query column sees, and the last steps of a row.
#pragma once
#include "cache_dev.h"

namespace jolt {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// The maximum of a part whose sum of weights is l: a part that met a NaN counts
// above every other, so that no join leaves it out as a part that saw nothing (its
// maximum may still be -infinity) or as one whose weights have vanished.
__device__ __forceinline__ float nan_outweighs(float m, float l) { return l != l ? 3e38f : m; }

// Which (sequence, KV head, columns, token range) a workgroup has.  Workgroups
// go to the 8 XCDs in turn; all of one (sequence, head) stay on one XCD, whose L2
// then serves its rows of the cache, and the units are dealt out one by one, so
// that sequences of unequal length spread over all XCDs.  Fewer than 32 units
// that 8 does not divide are left in plain order (some XCDs would stay idle).
struct AttnTile {
    int b, h, ct, split;
    bool valid;
};
__host__ __device__ __forceinline__ bool attn_by_xcd(int64_t units) { return units % 8 == 0 || units >= 32; }
__host__ __device__ __forceinline__ int64_t attn_grid(int64_t units, int64_t per) {
    return (attn_by_xcd(units) ? (units + 7) / 8 * 8 : units) * per;
}
__device__ __forceinline__ AttnTile attn_tile(const CacheAttnArgs &a, int ctiles) {
    const uint32_t units = (uint32_t)a.c.batch * a.c.H, per = (uint32_t)ctiles * a.splits, w = blockIdx.x;
    uint32_t u, in;
    if (attn_by_xcd(units)) {
        u = w / 8 / per * 8 + w % 8;
        in = w / 8 % per;
    } else {
        u = w / per;
        in = w % per;
    }
    AttnTile t;
    t.valid = u < units;
    t.b = u / a.c.H;
    t.h = u % a.c.H;
    t.ct = ctiles - 1 - in / a.splits;                 // later rows see more: they start first
    t.split = in % a.splits;
    return t;
}

// bits e = 0..7 set where lo <= tb + e < hi (all three in 0 .. 2^30 or, for lo, above)
__device__ __forceinline__ uint32_t range8(int tb, int lo, int hi) {
    const int h = min(max(hi - tb, 0), 8), l = min(max(lo - tb, 0), 8);
    return ((1u << h) - 1u) & (0xFFu << l);
}

// ancestors of a drafted token above itself
__device__ __forceinline__ int tree_depth(uint64_t mask) {
    const int n = (int)__popcll(mask);
    return n > 0 ? n - 1 : 0;
}

// What a query column may see: tokens of [first, kept) and of [lo, hi), and of a
// tree's slots (tokens from base on) those of its mask.
struct Column {
    int pos, first, kept, lo, hi;
    float slope;                          // slope * log2 e
    uint64_t mask;

    // column c of KV head h in sequence b (valid: c < n G), whose n rows start at s0
    __device__ __forceinline__ Column(const CacheAttnArgs &a, int s0, int n, int base, int len, int prefix, int h, int c,
                                      bool valid) {
        const int i = valid ? c / a.G : 0;
        mask = 0;
        pos = base + i;
        if (a.tree) {
            mask = valid ? a.tree[s0 + i] : 0;
            pos = base + tree_depth(mask);
            const int slots = min(min(n, kMaxKeep), len - base);
            mask &= slots >= 64 ? ~0ull : (slots > 0 ? (1ull << slots) - 1ull : 0ull);
            if (a.window > 0)             // a slot stands at the depth of its own path
                for (int j = 0; j < min(n, kMaxKeep); ++j)
                    if (tree_depth(a.tree[s0 + j]) <= pos - base - a.window) mask &= ~(1ull << j);
        }
        first = valid && a.first ? max(a.first[s0 + i], 0) : 0;
        kept = a.tree ? min(prefix, base) : min(prefix, len);
        lo = max(a.window > 0 ? pos - a.window + 1 : 0, first);
        hi = a.tree ? base : min(pos + 1, len);
        slope = a.slopes ? a.slopes[h * a.G + (valid ? c % a.G : 0)] * kLog2e : 0.f;
    }
    // which of tokens tb .. tb + 7 are visible
    __device__ __forceinline__ uint32_t sees8(bool tree, int base, int tb) const {
        uint32_t v = range8(tb, first, kept) | range8(tb, lo, hi);
        if (tree && tb + 8 > base) {
            const int s = tb - base;
            if (s < 64) v |= (uint32_t)(s >= 0 ? mask >> s : mask << -s) & 0xFFu;
        }
        return v;
    }
    // |position of this row - position of token t|
    __device__ __forceinline__ float distance(const CacheAttnArgs &a, int t, int s0, int n, int base) const {
        int tp = t;
        if (a.tree && t >= base && t - base < n) tp = base + tree_depth(a.tree[s0 + t - base]);
        return fabsf((float)(pos - tp));
    }
};

// Token ranges of a set of columns: [lo_any, hi_any) holds every token some
// column may see, apart from the prefix; every column sees all of [lo_all, hi_all).
struct Reach {
    int lo_any, hi_any, lo_all, hi_all, first_any;
    __device__ __forceinline__ Reach(const Column &c, bool valid) {
        lo_any = valid ? c.lo : 0x7FFFFFFF;
        hi_any = valid ? c.hi : 0;
        lo_all = valid ? c.lo : -0x7FFFFFFF;
        hi_all = valid ? c.hi : 0x7FFFFFFF;
        first_any = valid ? c.first : 0x7FFFFFFF;
    }
    // over aligned groups of W lanes
    template <int W>
    __device__ __forceinline__ void join() {
#pragma unroll
        for (int x = 1; x < W; x *= 2) {
            lo_any = min(lo_any, __shfl_xor(lo_any, x));
            hi_any = max(hi_any, __shfl_xor(hi_any, x));
            lo_all = max(lo_all, __shfl_xor(lo_all, x));
            hi_all = min(hi_all, __shfl_xor(hi_all, x));
            first_any = min(first_any, __shfl_xor(first_any, x));
        }
    }
    __device__ __forceinline__ void clip(const CacheAttnArgs &a, int len, int prefix) {
        if (a.tree) hi_any = len;
        hi_any = min(max(hi_any, prefix), len);
        hi_all = min(hi_all, len);
    }
    // the same in every lane: into scalar registers
    __device__ __forceinline__ void uniform() {
        lo_any = __builtin_amdgcn_readfirstlane(lo_any);
        hi_any = __builtin_amdgcn_readfirstlane(hi_any);
        lo_all = __builtin_amdgcn_readfirstlane(lo_all);
        hi_all = __builtin_amdgcn_readfirstlane(hi_all);
        first_any = __builtin_amdgcn_readfirstlane(first_any);
    }
    // the first token any column may see, the prefix included
    __device__ __forceinline__ int begin(int prefix) const {
        return max(prefix > first_any ? min(first_any, lo_any) : lo_any, 0);
    }
};

// The last steps of a row: its log-sum-exp and the weights of its own sums and of
// the part to be merged in.
struct RowEnd {
    float own, other, lse;
};
__device__ __forceinline__ RowEnd row_end(const CacheAttnArgs &a, int64_t at, float m, float l) {
    RowEnd r{1.f, 0.f, l == 0.f ? neg_inf() : (m + __builtin_amdgcn_logf(l)) * kLn2};
    if (a.merge_out) {
        const float l2 = a.merge_lse[at], mx = fmaxf(r.lse, l2);
        const float w1 = mx == neg_inf() ? 0.f : __builtin_amdgcn_exp2f((r.lse - mx) * kLog2e);
        const float w2 = mx == neg_inf() ? 0.f : __builtin_amdgcn_exp2f((l2 - mx) * kLog2e);
        const float s = w1 + w2, is = s == 0.f ? 0.f : 1.f / s;
        r.own = w1 * is;
        r.other = w2 * is;
        r.lse = s == 0.f ? neg_inf() : mx + __builtin_amdgcn_logf(s) * kLn2;
    }
    return r;
}
// 8 features from f on; a part that saw nothing adds nothing, whatever its rows hold
template <int D>
__device__ __forceinline__ void store_out8(const CacheAttnArgs &a, int64_t row, int head, int f, float (&o)[8], const RowEnd &r) {
    if (a.merge_out) {
        const float4 *p = reinterpret_cast<const float4 *>(a.merge_out + (row * a.hq + head) * D + f);
        const float4 x = p[0], y = p[1];
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (r.own == 0.f ? 0.f : o[e] * r.own) + (r.other == 0.f ? 0.f : v[e] * r.other);
    }
    uint16_t *dst = static_cast<uint16_t *>(a.out.ptr) + row * a.out.ts + head * a.out.hs + f;
    *reinterpret_cast<uint4 *>(dst) =
        make_uint4(bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]), bf16_pair(o[4], o[5]), bf16_pair(o[6], o[7]));
}

// out row: o (8 features of lane j of D/8), l and m (log2 domain) of the whole row
template <int D, bool ROT>
__device__ __forceinline__ void finish_row(const CacheAttnArgs &a, int64_t row, int head, int j, float (&o)[8], float m,
                                           float l, bool store) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= inv;
    if constexpr (ROT) {
        fwht_row<D>(o, j);
        const uint32_t sb = sign_byte(a.c.sv, j);
        const float isd = D == 128 ? 0.08838834764831845f : 0.125f;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = flip(o[e] * isd, (sb >> e) & 1);
    }
    if (!store) return;
    const int64_t at = row * a.hq + head;
    const RowEnd r = row_end(a, at, m, l);
    store_out8<D>(a, row, head, 8 * j, o, r);
    if (a.lse && j == 0) a.lse[at] = r.lse;
}

}  // namespace jolt
