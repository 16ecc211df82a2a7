// Token cache: page layout, argument checks (plain C++, no HIP) and the launch
// interface of its kernels (k_cache.hip, k_cache_attn.hip).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/libjolt.h"

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define JOLT_HD __host__ __device__ __forceinline__
#else
#define JOLT_HD inline
#endif

namespace jolt {

// One (page, head) block of the pool: K codes | V codes | K scales | V scales.
struct PageLayout {
    int64_t v_codes, k_scales, v_scales, bytes;      // offsets; K codes start at 0
};
JOLT_HD PageLayout page_layout(int page_tokens, int d, int bits) {
    PageLayout p;
    const int64_t codes = (int64_t)page_tokens * d * bits / 8, scales = (int64_t)page_tokens * (d / 64) * 2;
    p.v_codes = codes;
    p.k_scales = 2 * codes;
    p.v_scales = 2 * codes + scales;
    p.bytes = 2 * codes + 2 * scales;
    return p;
}

// What the kernels need of a jolt_cache.
struct CacheView {
    uint8_t *pool;
    const int32_t *table, *lens;
    int H, pages, max_pages, page_shift, batch;
    int64_t head_bytes;
    uint32_t sk[4], sv[4];                           // rotation signs (bit f set: s_f = -1)
};

// The pool page of token t of sequence b, or -1: past the table row, or a table
// entry that names no page of the pool.  Tokens of such pages are left out.
JOLT_HD int cache_page(const CacheView &c, int b, int t) {
    const int p = t >> c.page_shift;
    if (t < 0 || p >= c.max_pages) return -1;
    const int id = c.table[(size_t)b * c.max_pages + p];
    return (unsigned)id < (unsigned)c.pages ? id : -1;
}
JOLT_HD int64_t cache_block_offset(const CacheView &c, int page, int h) {
    return ((int64_t)page * c.H + h) * c.head_bytes;
}
// Rows starts[b] .. of a ragged call that belong to sequence b: none where the
// offsets do not increase or leave [0, total].
JOLT_HD int ragged_rows(const int32_t *starts, int b, int total, int *s0) {
    const int a = starts[b], e = starts[b + 1];
    *s0 = a;
    return (a >= 0 && e <= total && e > a) ? e - a : 0;
}
// lens[b] as the kernels use it: within the table row's capacity
JOLT_HD int cache_len(const CacheView &c, int b) {
    const int cap = c.max_pages << c.page_shift, l = c.lens[b];
    return l < 0 ? 0 : (l < cap ? l : cap);
}

// ---- checks (cache_args.cpp): JOLT_OK, or an error with its message in *msg
jolt_status cache_check(const jolt_cache *c, int32_t batch, const char **msg);
jolt_status rows_check(const jolt_rows *r, int64_t total, int heads, int d, int elem, bool output, const char **msg);
struct AttnPlan {
    bool wide;                                       // many query columns: k_cache_attn_wide
    int splits;                                      // token ranges a row's cache is cut into
    size_t ml_off, part_off, bytes;                  // workspace: [splits][rows][2], [splits][rows][d] fp32
};
jolt_status cache_attn_check(const jolt_cache *c, int32_t batch, int32_t total, int32_t max_q, int32_t max_len,
                             int32_t q_heads, const char **msg);
AttnPlan cache_attn_plan(const jolt_cache &c, int batch, int64_t total, int max_q, int max_len, int q_heads);
// least tokens of a range, for a window and max_len
int cache_attn_least(const AttnPlan &p, int max_q, int max_len, int window, bool prefix);
int page_shift_of(int page_tokens);

#if defined(__HIPCC__)
// ---- launches
struct RowsView {
    void *ptr;
    int64_t ts, hs;                                  // element strides of a token and of a head
};
// append / read: rows of `starts`, at most max_rows of a sequence
struct CacheRowsArgs {
    CacheView c;
    const int32_t *starts, *first;                   // first: read only (nullptr: 0)
    RowsView k, v;
    int total, max_rows;
};
hipError_t launch_cache_append(const CacheRowsArgs &a, int d, int bits, int dtype, bool rotate, hipStream_t s);
hipError_t launch_cache_read(const CacheRowsArgs &a, int d, int bits, int dtype, bool rotate, hipStream_t s);
struct CacheKeepArgs {
    CacheView c;
    const int32_t *base, *starts, *path;
    int total;
};
constexpr int kMaxKeep = 64;                         // path entries of a sequence, drafted tokens of a tree
hipError_t launch_cache_keep(const CacheKeepArgs &a, int d, int bits, hipStream_t s);

struct CacheAttnArgs {
    CacheView c;
    const int32_t *starts;
    RowsView q, out;
    float *lse;
    const float *slopes;
    const int32_t *prefix, *first;
    const uint64_t *tree;
    const float *merge_out, *merge_lse;
    float *ws_ml, *ws_part;
    float scale, cap;
    int window, total, max_q, hq, G, splits, least;
};
hipError_t launch_cache_attention(const CacheAttnArgs &a, bool wide, int d, int bits, bool rotate, hipStream_t s);
hipError_t launch_cache_attn_wide(const CacheAttnArgs &a, int d, int bits, bool rotate, hipStream_t s);
#endif

}  // namespace jolt
