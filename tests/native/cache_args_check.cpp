// Drives the token cache's host checks (csrc/cache_args.cpp) and its index
// helpers (csrc/cache.h) with valid, refused and random arguments.  Prints
// "cache args: N failures".
#include <cstdio>
#include <random>
#include <vector>

#include "cache.h"

using namespace jolt;

static int failures = 0;
#define EXPECT(c)                                                  \
    do {                                                           \
        if (!(c)) {                                                \
            std::printf("line %d: %s\n", __LINE__, #c);            \
            ++failures;                                            \
        }                                                          \
    } while (0)

static jolt_cache good(std::vector<uint8_t> &pool, std::vector<int32_t> &table, std::vector<int32_t> &lens) {
    jolt_cache c{};
    c.H = 2; c.d = 128; c.bits = 4; c.page_tokens = 64; c.pages = 5; c.max_pages = 3;
    pool.assign(page_layout(64, 128, 4).bytes * 2 * 5 + 16, 0);
    table.assign(2 * 3, 0);
    lens.assign(2, 0);
    c.pool = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(pool.data()) + 15) / 16 * 16);
    c.pool_bytes = page_layout(64, 128, 4).bytes * 2 * 5;
    c.table = table.data();
    c.lens = lens.data();
    return c;
}

int main() {
    std::vector<uint8_t> pool;
    std::vector<int32_t> table, lens;
    const jolt_cache g = good(pool, table, lens);
    const char *msg = "";
    EXPECT(cache_check(&g, 2, &msg) == JOLT_OK);
    EXPECT(cache_check(nullptr, 2, &msg) == JOLT_E_INVALID);
    auto with = [&](auto set, int batch = 2) {
        jolt_cache c = g;
        set(c);
        return cache_check(&c, batch, &msg);
    };
    EXPECT(with([](jolt_cache &c) { c.d = 96; }) == JOLT_E_UNSUPPORTED);
    EXPECT(with([](jolt_cache &c) { c.bits = 3; }) == JOLT_E_UNSUPPORTED);
    for (int p : {0, 1, 16, 48, 512, -64}) EXPECT(with([p](jolt_cache &c) { c.page_tokens = p; }) == JOLT_E_UNSUPPORTED);
    EXPECT(with([](jolt_cache &c) { c.H = 0; }) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &c) { c.pages = -1; }) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &c) { c.max_pages = -1; }) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &c) { c.max_pages = 1 << 25; }) == JOLT_E_UNSUPPORTED);
    EXPECT(with([](jolt_cache &c) { c.table = nullptr; }) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &c) { c.lens = nullptr; }) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &c) { c.pool = nullptr; }) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &c) { c.pool = static_cast<uint8_t *>(c.pool) + 8; }) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &c) { c.pool_bytes -= 1; }) == JOLT_E_WORKSPACE);
    EXPECT(with([](jolt_cache &c) { c.pages = 0x7FFFFFFF; }) == JOLT_E_WORKSPACE);
    EXPECT(with([](jolt_cache &) {}, -1) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &) {}, 1 << 24) == JOLT_E_INVALID);
    EXPECT(with([](jolt_cache &c) { c.pool = nullptr; c.lens = nullptr; c.table = nullptr; }, 0) == JOLT_OK);

    alignas(16) static uint8_t buf[64];
    auto rows = [&](void *p, int64_t ts, int64_t hs, int64_t total, int heads, bool out, int elem = 2) {
        jolt_rows r{p, ts, hs};
        return rows_check(&r, total, heads, 128, elem, out, &msg);
    };
    EXPECT(rows(buf, 1024, 128, 7, 8, true) == JOLT_OK);           // token-major
    EXPECT(rows(buf, 128, 7 * 128, 7, 8, true) == JOLT_OK);        // head-major
    EXPECT(rows(buf, 4096, 256, 7, 8, true) == JOLT_OK);           // padded
    EXPECT(rows(buf, 1016, 128, 7, 8, true) == JOLT_E_INVALID);    // rows overlap
    EXPECT(rows(buf, 1024, 64, 7, 8, true) == JOLT_E_INVALID);
    EXPECT(rows(buf, 0, 128, 7, 8, true) == JOLT_E_INVALID);
    EXPECT(rows(buf, 0, 128, 7, 8, false) == JOLT_OK);             // an input may repeat a row
    EXPECT(rows(buf, 1024, 0, 7, 1, true) == JOLT_OK);             // one head: its stride does not matter
    EXPECT(rows(buf, 0, 128, 1, 8, true) == JOLT_OK);
    EXPECT(rows(buf, 1025, 128, 7, 8, false) == JOLT_E_INVALID);   // 16 bytes
    EXPECT(rows(buf, 1028, 128, 7, 8, false) == JOLT_E_INVALID);
    EXPECT(rows(buf, 1028, 128, 7, 8, false, 4) == JOLT_OK);
    EXPECT(rows(buf + 2, 1024, 128, 7, 8, false) == JOLT_E_INVALID);
    EXPECT(rows(buf, -1024, 128, 7, 8, false) == JOLT_E_INVALID);
    EXPECT(rows(buf, (int64_t)1 << 62, 128, 7, 8, false) == JOLT_E_INVALID);
    EXPECT(rows(nullptr, 1024, 128, 7, 8, false) == JOLT_E_INVALID);
    EXPECT(rows(nullptr, 1024, 128, 0, 8, false) == JOLT_OK);
    EXPECT(rows_check(nullptr, 3, 8, 128, 2, false, &msg) == JOLT_E_INVALID);

    EXPECT(cache_attn_check(&g, 2, 10, 5, 100, 8, &msg) == JOLT_OK);
    EXPECT(cache_attn_check(&g, 2, 10, 5, 100, 3, &msg) == JOLT_E_INVALID);
    EXPECT(cache_attn_check(&g, 2, 10, 5, 100, 0, &msg) == JOLT_E_INVALID);
    EXPECT(cache_attn_check(&g, 2, -1, 5, 100, 8, &msg) == JOLT_E_INVALID);
    EXPECT(cache_attn_check(&g, 2, 10, -1, 100, 8, &msg) == JOLT_E_INVALID);
    EXPECT(cache_attn_check(&g, 2, 10, 5, -1, 8, &msg) == JOLT_E_INVALID);
    EXPECT(cache_attn_check(&g, 2, 0x7FFFFFFF, 5, 100, 8, &msg) == JOLT_E_UNSUPPORTED);
    EXPECT(cache_attn_check(&g, 2, 10, 0x7FFFFFFF, 100, 8, &msg) == JOLT_E_UNSUPPORTED);

    // page lookups stay inside the table row and the pool, whatever the table holds
    std::mt19937 rng(1);
    for (int it = 0; it < 20000; ++it) {
        CacheView v{};
        v.H = 1 + rng() % 3;
        v.pages = rng() % 6;
        v.max_pages = rng() % 5;
        v.page_shift = 5 + rng() % 4;
        v.batch = 1 + rng() % 3;
        v.head_bytes = page_layout(1 << v.page_shift, 64, 4).bytes;
        std::vector<int32_t> t((size_t)v.batch * v.max_pages);
        for (auto &x : t) x = (int)(rng() % 12) - 4;
        if (!t.empty() && rng() % 4 == 0) t[rng() % t.size()] = (int32_t)rng();
        std::vector<int32_t> l(v.batch);
        for (auto &x : l) x = (rng() % 3) ? (int)(rng() % 3000) - 500 : (int32_t)rng();
        v.table = t.data();
        v.lens = l.data();
        const int b = rng() % v.batch;
        const int tok = (rng() % 8) ? (int)(rng() % 3000) - 100 : (int32_t)rng();
        const int p = cache_page(v, b, tok);
        EXPECT(p >= -1 && p < v.pages);
        if (p >= 0) {
            const int64_t o = cache_block_offset(v, p, v.H - 1);
            EXPECT(o >= 0 && o + v.head_bytes <= v.head_bytes * v.H * v.pages);
        }
        const int len = cache_len(v, b);
        EXPECT(len >= 0 && len <= (v.max_pages << v.page_shift));
        int32_t st[2] = {(rng() % 4) ? (int)(rng() % 12) - 2 : (int32_t)rng(), (rng() % 4) ? (int)(rng() % 12) - 2 : (int32_t)rng()};
        int s0;
        const int n = ragged_rows(st, 0, 9, &s0);
        EXPECT(n >= 0 && (n == 0 || (s0 >= 0 && s0 + n <= 9)));
    }
    // offsets past 32 bits
    CacheView big{};
    big.H = 8;
    big.head_bytes = page_layout(256, 128, 8).bytes;
    EXPECT(cache_block_offset(big, 200000, 7) == ((int64_t)200000 * 8 + 7) * big.head_bytes);
    std::printf("cache args: %d failures\n", failures);
    return failures != 0;
}
