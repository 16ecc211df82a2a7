// libjolt C ABI: the token cache's entry points.  Arguments are checked on the
// host (cache_args.cpp); what the device arrays hold is bounds-checked by the
// kernels.
#include <cmath>

#include "api_internal.h"
#include "cache.h"
#include "jolt_internal.h"

using namespace jolt;

namespace jolt {

// The handle's device for the time of a call, the caller's before and after.
class DeviceScope {
  public:
    explicit DeviceScope(int device) {
        if (hipGetDevice(&prev_) != hipSuccess) prev_ = -1;
        if (prev_ != device) err_ = hipSetDevice(device);
        else prev_ = -1;
    }
    ~DeviceScope() {
        if (prev_ >= 0) (void)hipSetDevice(prev_);
    }
    DeviceScope(const DeviceScope &) = delete;
    DeviceScope &operator=(const DeviceScope &) = delete;
    hipError_t error() const { return err_; }

  private:
    int prev_ = -1;
    hipError_t err_ = hipSuccess;
};

static CacheView view_of(const jolt_cache &c, int batch) {
    CacheView v{};
    v.pool = static_cast<uint8_t *>(c.pool);
    v.table = c.table;
    v.lens = c.lens;
    v.H = c.H;
    v.pages = c.pages;
    v.max_pages = c.max_pages;
    v.page_shift = page_shift_of(c.page_tokens);
    v.batch = batch;
    v.head_bytes = page_layout(c.page_tokens, c.d, c.bits).bytes;
    if (c.rotate) {
        sign_bits_for(c.seed, c.k_item_id, c.d, v.sk);
        sign_bits_for(c.seed, c.v_item_id, c.d, v.sv);
    }
    return v;
}

static RowsView rows_of(const jolt_rows &r) { return RowsView{r.ptr, r.token_stride, r.head_stride}; }

template <typename F>
static jolt_status guarded(jolt_handle h, F &&f) {
    if (!h) return JOLT_E_INVALID;
    try {
        clear_err(h);
        return f();
    } catch (...) {
        return JOLT_E_DEVICE;
    }
}

static jolt_status rows_call(jolt_handle h, bool read, const jolt_cache *cache, int32_t batch, const int32_t *first,
                             const int32_t *starts, int32_t total, int32_t max_rows, int32_t dtype, const jolt_rows *k,
                             const jolt_rows *v, void *stream) {
    const char *msg = "";
    jolt_status s = cache_check(cache, batch, &msg);
    if (s) return fail(h, s, "%s", msg);
    if (dtype != JOLT_BF16 && dtype != JOLT_F32) return fail(h, JOLT_E_INVALID, "cache: unknown dtype");
    if (total < 0 || max_rows < 0) return fail(h, JOLT_E_INVALID, "cache: negative row count");
    if (batch > 0 && !starts) return fail(h, JOLT_E_INVALID, "cache: NULL starts");
    const int elem = dtype == JOLT_F32 ? 4 : 2;
    if ((s = rows_check(k, total, cache->H, cache->d, elem, read, &msg))) return fail(h, s, "k: %s", msg);
    if ((s = rows_check(v, total, cache->H, cache->d, elem, read, &msg))) return fail(h, s, "v: %s", msg);
    if (batch == 0 || total == 0 || max_rows == 0) return JOLT_OK;
    if (((int64_t)max_rows / 8 + 2) * cache->H * batch > 0x7FFFFFFF)
        return fail(h, JOLT_E_UNSUPPORTED, "cache: too many rows for one call");
    DeviceScope dev(handle_device(h));
    if (dev.error() != hipSuccess) return hip_fail(h, dev.error(), "device");
    CacheRowsArgs a{};
    a.c = view_of(*cache, batch);
    a.starts = starts;
    a.first = first;
    a.k = rows_of(*k);
    a.v = rows_of(*v);
    a.total = total;
    a.max_rows = max_rows;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = read ? launch_cache_read(a, cache->d, cache->bits, dtype, cache->rotate != 0, st)
                              : launch_cache_append(a, cache->d, cache->bits, dtype, cache->rotate != 0, st);
    return e == hipSuccess ? JOLT_OK : hip_fail(h, e, read ? "cache_read" : "cache_append");
}

static jolt_status attn_call(jolt_handle h, const jolt_cache *cache, int32_t batch, const int32_t *starts, int32_t total,
                             int32_t max_q, int32_t max_len, int32_t q_heads, const jolt_rows *q, const uint64_t *tree,
                             const jolt_attn_terms *terms, const jolt_rows *out, float *lse, void *workspace,
                             size_t workspace_bytes, void *stream) {
    const char *msg = "";
    jolt_status s = cache_attn_check(cache, batch, total, max_q, max_len, q_heads, &msg);
    if (s) return fail(h, s, "%s", msg);
    if (!terms) return fail(h, JOLT_E_INVALID, "attention: NULL terms");
    if (!(terms->scale > 0.f) || !std::isfinite(terms->scale))
        return fail(h, JOLT_E_INVALID, "attention: scale must be > 0");
    if (!(terms->cap >= 0.f) || !std::isfinite(terms->cap)) return fail(h, JOLT_E_INVALID, "attention: cap must be >= 0");
    // what the kernels multiply scores with, in log2 units and in the cap's
    constexpr float kTwoLog2e = 2.8853901f;
    if (!std::isfinite(terms->scale * kTwoLog2e) ||
        (terms->cap > 0.f && (!std::isfinite(terms->scale / terms->cap * kTwoLog2e) || !std::isfinite(terms->cap * kTwoLog2e))))
        return fail(h, JOLT_E_INVALID, "attention: scale, cap or scale / cap is beyond fp32");
    if (terms->window < 0) return fail(h, JOLT_E_INVALID, "attention: window must be >= 0");
    if (!terms->merge_out != !terms->merge_lse)
        return fail(h, JOLT_E_INVALID, "attention: merge_out and merge_lse go together");
    if (reinterpret_cast<uintptr_t>(terms->merge_out) % 16)
        return fail(h, JOLT_E_INVALID, "attention: merge_out must be 16-byte aligned");
    if (batch > 0 && !starts) return fail(h, JOLT_E_INVALID, "attention: NULL starts");
    if ((s = rows_check(q, total, q_heads, cache->d, 2, false, &msg))) return fail(h, s, "q: %s", msg);
    if ((s = rows_check(out, total, q_heads, cache->d, 2, true, &msg))) return fail(h, s, "out: %s", msg);
    if (batch == 0 || total == 0 || max_q == 0) return JOLT_OK;
    const AttnPlan p = cache_attn_plan(*cache, batch, total, max_q, max_len, q_heads);
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes || reinterpret_cast<uintptr_t>(workspace) % 16))
        return fail(h, JOLT_E_WORKSPACE, "attention workspace: need %zu bytes (16-byte aligned), have %zu", p.bytes,
                    workspace_bytes);
    DeviceScope dev(handle_device(h));
    if (dev.error() != hipSuccess) return hip_fail(h, dev.error(), "device");
    CacheAttnArgs a{};
    a.c = view_of(*cache, batch);
    a.starts = starts;
    a.q = rows_of(*q);
    a.out = rows_of(*out);
    a.lse = lse;
    a.slopes = terms->slopes;
    a.prefix = terms->prefix;
    a.first = terms->first;
    a.tree = tree;
    a.merge_out = terms->merge_out;
    a.merge_lse = terms->merge_lse;
    a.ws_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + p.ml_off);
    a.ws_part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + p.part_off);
    a.scale = terms->scale;
    a.cap = terms->cap;
    a.window = terms->window;
    a.total = total;
    a.max_q = max_q;
    a.hq = q_heads;
    a.G = q_heads / cache->H;
    a.splits = p.splits;
    a.least = cache_attn_least(p, max_q, max_len, terms->window, terms->prefix != nullptr);
    const hipError_t e = launch_cache_attention(a, p.wide, cache->d, cache->bits, cache->rotate != 0,
                                                static_cast<hipStream_t>(stream));
    return e == hipSuccess ? JOLT_OK : hip_fail(h, e, "cache_attention");
}

}  // namespace jolt

extern "C" jolt_status jolt_cache_pool_bytes(const jolt_cache *cache, size_t *bytes) {
    if (!bytes) return JOLT_E_INVALID;
    jolt_status s = cache_check(cache, 0, nullptr);
    if (s) return s;
    *bytes = (size_t)(page_layout(cache->page_tokens, cache->d, cache->bits).bytes * cache->H) * cache->pages;
    return JOLT_OK;
}

extern "C" jolt_status jolt_cache_append(jolt_handle h, const jolt_cache *cache, int32_t batch, const int32_t *starts,
                                         int32_t total, int32_t max_new, int32_t dtype, const jolt_rows *k,
                                         const jolt_rows *v, void *stream) {
    return guarded(h, [&] {
        return rows_call(h, false, cache, batch, nullptr, starts, total, max_new, dtype, k, v, stream);
    });
}

extern "C" jolt_status jolt_cache_read(jolt_handle h, const jolt_cache *cache, int32_t batch, const int32_t *first,
                                       const int32_t *starts, int32_t total, int32_t max_rows, int32_t dtype,
                                       const jolt_rows *k, const jolt_rows *v, void *stream) {
    return guarded(h, [&] {
        return rows_call(h, true, cache, batch, first, starts, total, max_rows, dtype, k, v, stream);
    });
}

extern "C" jolt_status jolt_cache_keep(jolt_handle h, const jolt_cache *cache, int32_t batch, const int32_t *base,
                                       const int32_t *starts, const int32_t *path, int32_t total, void *stream) {
    return guarded(h, [&]() -> jolt_status {
        const char *msg = "";
        jolt_status s = cache_check(cache, batch, &msg);
        if (s) return fail(h, s, "%s", msg);
        if (total < 0 || (batch > 0 && total > 0 && (!base || !starts || !path)))
            return fail(h, JOLT_E_INVALID, "cache_keep: bad arguments");
        if (batch == 0 || total == 0) return JOLT_OK;
        if ((int64_t)batch * cache->H > 0x7FFFFFFF)
            return fail(h, JOLT_E_UNSUPPORTED, "cache_keep: too many sequences for one call");
        DeviceScope dev(handle_device(h));
        if (dev.error() != hipSuccess) return hip_fail(h, dev.error(), "device");
        CacheKeepArgs a{};
        a.c = view_of(*cache, batch);
        a.base = base;
        a.starts = starts;
        a.path = path;
        a.total = total;
        const hipError_t e = launch_cache_keep(a, cache->d, cache->bits, static_cast<hipStream_t>(stream));
        return e == hipSuccess ? JOLT_OK : hip_fail(h, e, "cache_keep");
    });
}

extern "C" jolt_status jolt_cache_attention_workspace_size(const jolt_cache *cache, int32_t batch, int32_t total,
                                                           int32_t max_q, int32_t max_len, int32_t q_heads,
                                                           size_t *bytes) {
    if (!bytes) return JOLT_E_INVALID;
    jolt_status s = cache_attn_check(cache, batch, total, max_q, max_len, q_heads, nullptr);
    if (s) return s;
    *bytes = batch == 0 || total == 0 || max_q == 0
                 ? 0 : cache_attn_plan(*cache, batch, total, max_q, max_len, q_heads).bytes;
    return JOLT_OK;
}

extern "C" jolt_status jolt_cache_attention(jolt_handle h, const jolt_cache *cache, int32_t batch, const int32_t *starts,
                                            int32_t total, int32_t max_q, int32_t max_len, int32_t q_heads,
                                            const jolt_rows *q, const jolt_attn_terms *terms, const jolt_rows *out,
                                            float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    return guarded(h, [&] {
        return attn_call(h, cache, batch, starts, total, max_q, max_len, q_heads, q, nullptr, terms, out, lse,
                         workspace, workspace_bytes, stream);
    });
}

extern "C" jolt_status jolt_tree_attention(jolt_handle h, const jolt_cache *cache, int32_t batch, const int32_t *starts,
                                           int32_t total, int32_t max_q, int32_t max_len, int32_t q_heads,
                                           const jolt_rows *q, const uint64_t *tree, const jolt_attn_terms *terms,
                                           const jolt_rows *out, float *lse, void *workspace, size_t workspace_bytes,
                                           void *stream) {
    return guarded(h, [&]() -> jolt_status {
        if (max_q > kMaxKeep) return fail(h, JOLT_E_UNSUPPORTED, "tree: at most 64 drafted tokens of a sequence");
        if (total > 0 && !tree) return fail(h, JOLT_E_INVALID, "tree: NULL masks");
        return attn_call(h, cache, batch, starts, total, max_q, max_len, q_heads, q, tree, terms, out, lse, workspace,
                         workspace_bytes, stream);
    });
}
