// Token cache: argument checks and sizes.  Plain C++ (no HIP), so that the
// checks also build and run on their own on the host.
#include "cache.h"

#include <algorithm>
#include <limits>

namespace jolt {

int page_shift_of(int page_tokens) {
    for (int s = 5; s <= 8; ++s)
        if (page_tokens == (1 << s)) return s;
    return -1;
}

static jolt_status refuse(const char **msg, jolt_status s, const char *text) {
    if (msg) *msg = text;
    return s;
}

jolt_status cache_check(const jolt_cache *c, int32_t batch, const char **msg) {
    if (!c) return refuse(msg, JOLT_E_INVALID, "cache: NULL");
    if (c->d != 64 && c->d != 128) return refuse(msg, JOLT_E_UNSUPPORTED, "cache: d must be 64 or 128");
    if (c->bits != 4 && c->bits != 8) return refuse(msg, JOLT_E_UNSUPPORTED, "cache: bits must be 4 or 8");
    if (page_shift_of(c->page_tokens) < 0)
        return refuse(msg, JOLT_E_UNSUPPORTED, "cache: page_tokens must be 32, 64, 128 or 256");
    if (c->H < 1 || c->H > 65535) return refuse(msg, JOLT_E_INVALID, "cache: H must be 1..65535");
    if (c->pages < 0 || c->max_pages < 0) return refuse(msg, JOLT_E_INVALID, "cache: negative page count");
    if ((int64_t)c->max_pages * c->page_tokens > std::numeric_limits<int32_t>::max() / 2)
        return refuse(msg, JOLT_E_UNSUPPORTED, "cache: more than 2^30 tokens in a sequence");
    if (batch < 0 || batch > (1 << 20)) return refuse(msg, JOLT_E_INVALID, "cache: batch must be 0..2^20");
    if (batch > 0) {
        if (!c->lens || (c->max_pages > 0 && !c->table)) return refuse(msg, JOLT_E_INVALID, "cache: NULL table or lens");
        if (c->pages > 0 && !c->pool) return refuse(msg, JOLT_E_INVALID, "cache: NULL pool");
        if (reinterpret_cast<uintptr_t>(c->pool) % 16)
            return refuse(msg, JOLT_E_INVALID, "cache: the pool must be 16-byte aligned");
        const uint64_t page = (uint64_t)page_layout(c->page_tokens, c->d, c->bits).bytes * c->H;
        if (c->pool_bytes / page < (uint64_t)c->pages) return refuse(msg, JOLT_E_WORKSPACE, "cache: pool smaller than its pages");
    }
    return JOLT_OK;
}

// Row views: 16-byte aligned rows; an output's rows must not overlap (token- or
// head-major, or padded forms of these).
jolt_status rows_check(const jolt_rows *r, int64_t total, int heads, int d, int elem, bool output, const char **msg) {
    if (total == 0) return JOLT_OK;
    if (!r || !r->ptr) return refuse(msg, JOLT_E_INVALID, "rows: NULL");
    const int64_t unit = 16 / elem;
    if (reinterpret_cast<uintptr_t>(r->ptr) % 16 || r->token_stride % unit || r->head_stride % unit)
        return refuse(msg, JOLT_E_INVALID, "rows: pointer and strides must be multiples of 16 bytes");
    if (r->token_stride < 0 || r->head_stride < 0) return refuse(msg, JOLT_E_INVALID, "rows: negative stride");
    const int64_t lim = std::numeric_limits<int64_t>::max() / 16 / std::max<int64_t>(std::max<int64_t>(total, heads), 1);
    if (r->token_stride > lim || r->head_stride > lim) return refuse(msg, JOLT_E_INVALID, "rows: stride too large");
    if (output) {
        const int64_t ts = r->token_stride, hs = r->head_stride;
        const bool token_major = (total == 1 || ts >= (heads - 1) * hs + d) && (heads == 1 || hs >= d);
        const bool head_major = (heads == 1 || hs >= (total - 1) * ts + d) && (total == 1 || ts >= d);
        if (!token_major && !head_major) return refuse(msg, JOLT_E_INVALID, "rows: output rows overlap");
    }
    return JOLT_OK;
}

jolt_status cache_attn_check(const jolt_cache *c, int32_t batch, int32_t total, int32_t max_q, int32_t max_len,
                             int32_t q_heads, const char **msg) {
    jolt_status s = cache_check(c, batch, msg);
    if (s) return s;
    if (total < 0 || max_q < 0 || max_len < 0) return refuse(msg, JOLT_E_INVALID, "attention: negative size");
    if (q_heads < c->H || q_heads % c->H || q_heads > 65535)
        return refuse(msg, JOLT_E_INVALID, "attention: q_heads must be a multiple of H, at most 65535");
    const int64_t tiles = (int64_t)batch * c->H * (((int64_t)max_q * (q_heads / c->H) + 15) / 16);
    if (tiles > (1 << 24) || (int64_t)total * q_heads > std::numeric_limits<int32_t>::max() / 2)
        return refuse(msg, JOLT_E_UNSUPPORTED, "attention: too many query rows for one call");
    return JOLT_OK;
}

// Narrow kernel (tiles of 16 query columns of a KV head and sequence, 4 waves) or
// wide one (tiles of 256, one per CU).  The wide one computes a score for a third
// less where it is busy, but its start and end cost 17 us against 8, and a tile
// that is not full costs what a full one does.  8 heads, d = 128, 4 bits, narrow
// against wide in us: 16 x 4096 tokens 116 : 127 at 128 columns, 145 : 129 at 160,
// 221 : 138 at 256; 16 x 1024 tokens 56 : 56 at 192 columns; 16384 tokens 52 : 55
// at 192 and 62 : 61 at 256; 4096 tokens 26 : 44 at 256.  So the wide one takes
// more than 128 columns with more than 24 * 2^20 scores.
// Token ranges: enough workgroups for the 256 CUs (two of the narrow kernel's share
// one), none of fewer than 256 tokens (wide: 512).  A decode step in ranges of at
// least 128, 256 and 512 tokens: 11.1, 11.4, 13.7 us at 1024 tokens, 14.4, 12.6
// us at 4 x 2048 (128, 256); wide, 256 and 512 tokens: 60.9 and 59.9 us at 16384.
AttnPlan cache_attn_plan(const jolt_cache &c, int batch, int64_t total, int max_q, int max_len, int q_heads) {
    AttnPlan p{};
    const int64_t cols = (int64_t)max_q * (q_heads / c.H);
    p.wide = cols > 128 && (double)batch * c.H * cols * max_len > 24.0 * (1 << 20);
    const int64_t per = p.wide ? 256 : 16, want = p.wide ? 256 : 512, least = p.wide ? 512 : 256;
    const int64_t tiles = std::max<int64_t>(1, (int64_t)batch * c.H * ((cols + per - 1) / per));
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(max_len / least, want / tiles), 256));
    if (p.splits > 1) {
        const size_t rows = (size_t)total * q_heads;
        p.ml_off = 0;
        p.part_off = (p.splits * rows * 2 * 4 + 255) / 256 * 256;
        p.bytes = p.part_off + p.splits * rows * c.d * 4;
    }
    return p;
}

// A sequence shorter than the longest is cut into fewer ranges of the longest
// one's size, not into as many small ones, so that a ragged batch's ranges take
// equal time.
int cache_attn_least(const AttnPlan &p, int max_q, int max_len, int window, bool prefix) {
    int64_t seen = max_len;
    if (window > 0 && !prefix) seen = std::min<int64_t>(seen, (int64_t)window + max_q);
    return (int)((seen + p.splits - 1) / p.splits);
}

}  // namespace jolt
