// Attention over the token cache for many query rows (prompt chunks, trees):
// the same sums as k_cache_attn.hip, with 64-token tiles of the cache put into LDS
// once per workgroup and shared by its 8 waves of 32 query columns.
//
// On the way to LDS the quantization is undone, so that a score costs one product
// and no scaling: rows are held in fp16 as q sc 2^-E, with E a scale exponent of
// the tile.  For 4-bit codes that is exact (3 + 8 significant bits) down to 2^-18
// of the tile's largest scale; for 8-bit ones K holds the codes alone (their scales
// multiply the scores of each group of 64 in fp32) and V is rounded to fp16
// (2^-11).  E of K is its largest scale's; E of V is kept from tile to tile while
// it fits, because the sums are in its unit.  A tile whose scales lie further
// apart, or jump, is "wild": every token has a unit of its own there, kept beside
// the tile, which multiplies its scores and weights, and each column's sum changes
// to the unit that its largest weight asks for.
// Queries are divided by a power of two that brings their largest feature to [1, 2)
// and held in fp16: exact for bf16 queries (below 2^-16 of the largest, to 2^-25 of
// it), two parts (2^-22) for rotated ones (one part alone takes a fifth off the
// time, and puts 5e-6 on the log-sum-exp where two leave 3e-7).  Weights are rounded
// to fp16 (2^-11); what falls below 2^-24 of the column's largest is lost.
//
// Products are S^T = K Q^T and O^T = V^T P^T in 32x32x16, and as in the narrow
// kernel a lane's scores are, in order, its operand of the second product.
//
// LDS (158 KB at d = 128, rotated): two K buffers, three V buffers, the queries'
// second parts, the columns' limits; the first parts, the sums, scores and weights
// are in registers (227-256 a lane), so a CU holds one workgroup, two waves a SIMD.
//
// Bound by the matrix unit and the vector unit in turn: 2048 rows x 32 heads at the
// end of 8192 tokens, d = 128, 4 bits, rotated: 348 us, 689 TFLOP/s of plain
// attention and 1.5 times that in products (matrix pipes busy 56 % of the cycles;
// a large bf16 product reaches 1240 TFLOP/s).  A turn of products takes about 2700
// cycles where its 48 instructions need 1536, a turn of softmax and units 2400.
// Measured steps: 8 waves without turns 412 us; turns 375; tiles and loads between
// the products and s_setprio 348.  48 drafted rows x 32 heads of 16 sequences over
// 4144 tokens 96 us (192 of 256 columns are there); 4 x 509 packed rows of 40 heads,
// window 1024, 8 bits 72 us (320 workgroups on 256 CUs, of which 17 us is each one's
// start and end).
#include <algorithm>

#include "cache.h"
#include "cache_attn_dev.h"
#include "jolt_internal.h"
#include "ktimer.h"

namespace jolt {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;                              // tokens of a tile

__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}
__device__ __forceinline__ f16x2 h2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }
__device__ __forceinline__ uint32_t u32(f16x2 v) { return __builtin_bit_cast(uint32_t, v); }

// a unit of 8 codes as signed fp16 integers, exact.  4 bits: a nibble under the
// exponent of 1024 is 1024 + u, or 1024 + 16 u from the next nibble up.  `magic`
// is 0x64006400 in a vector register (with the mask in a scalar one, an and-or
// is one instruction).
template <int BITS>
__device__ __forceinline__ void unit_f16(const uint32_t *w, uint32_t magic, f16x2 (&x)[4]) {
    if constexpr (BITS == 4) {
        const f16x2 c0 = {(_Float16)-1032.f, (_Float16)-1032.f}, c1 = {(_Float16)-72.f, (_Float16)-72.f};
        const f16x2 r = {(_Float16)0.0625f, (_Float16)0.0625f};
        uint32_t m0 = 0x000F000Fu, m1 = 0x00F000F0u;
        asm("" : "+s"(m0), "+s"(m1));
        const uint32_t a = w[0], b = a >> 8;
        x[0] = h2((a & m0) | magic) + c0;
        x[1] = __builtin_elementwise_fma(h2((a & m1) | magic), r, c1);
        x[2] = h2((b & m0) | magic) + c0;
        x[3] = __builtin_elementwise_fma(h2((b & m1) | magic), r, c1);
    } else {
        const f16x2 c0 = {(_Float16)-1152.f, (_Float16)-1152.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)                    // bytes 2 i, 2 i + 1 under the exponent of 1024
            x[i] = h2(__builtin_amdgcn_perm(w[i >> 1], magic, (i & 1) ? 0x01070106u : 0x01050104u)) + c0;
    }
}

// two bf16 scales as fp16 with their exponent fields lowered by `down` (of both
// halves, at bit 7); what falls below the range becomes 0
__device__ __forceinline__ f16x2 scale_f16(uint32_t two, uint32_t down) {
    const u16x2 v = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, two), __builtin_bit_cast(u16x2, down));
    return __builtin_bit_cast(f16x2, v << u16x2{3, 3});
}
__device__ __forceinline__ uint32_t pk_umax(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
template <int Ctrl>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, Ctrl, 0xF, 0xF, false);
}

// two +-1 in bf16: the signs of H at (f, c) and (f, c + 1), c even
__device__ __forceinline__ uint32_t sign_ones(uint32_t f, uint32_t c) {
    const uint32_t p = __popc(f & c) & 1;
    return 0x3F803F80u ^ (p << 15) ^ ((p ^ (f & 1)) << 31);
}
// the fragment with these signs over its elements and parity(f & c) for all
__device__ __forceinline__ bf16x8 sign_frag(const uint32_t (&b)[4], uint32_t f, uint32_t c) {
    const uint32_t all = (__popc(f & c) & 1) ? 0x80008000u : 0u;
    return __builtin_bit_cast(bf16x8, make_uint4(b[0] ^ all, b[1] ^ all, b[2] ^ all, b[3] ^ all));
}
// bits e and e + 1 of s as the signs of a bf16 pair
__device__ __forceinline__ uint32_t sign_pair(uint32_t s, int e) {
    const uint32_t two = s >> e;
    return ((two & 1u) << 15) | ((two & 2u) << 30);
}

// One thread's share of a tile: UPT units of K and of V and the scales they
// need; all: two scales a lane of each half of the tile (lanes 0..31 K, 32..63
// V), for the tile's largest.
template <int D, int BITS, int NT>
struct TileRegs {
    static constexpr int kU = BITS / 4;                // dwords of a unit
    static constexpr int UPT = kTile * D / 8 / NT;
    static constexpr int FS = NT / 8;                  // a thread's V features: f, f + FS, ...
    uint32_t k[UPT * kU], v[UPT * kU], vs[D / 64][4], all[2];
    uint16_t ks[D / 64];
};

}  // namespace

template <int D, int BITS, bool ROT, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_cache_attn_wide(CacheAttnArgs a, int ctiles) {
    constexpr int NT = 64 * NW, NK = D / 16, NF = D / 32, NG = D / 64;
    constexpr bool kPost = BITS == 8;                  // K scales multiply the scores
    constexpr int kTop = BITS == 4 ? 27 : 23;          // fp16 exponent field of the largest scale
    constexpr int kKStride = kTile * 16 + 32;          // bytes of a K chunk (8 features of 64 tokens), padded
    constexpr int kKBytes = D / 8 * kKStride, kVBytes = kTile / 8 * D * 16;
    constexpr int kSBytes = kPost ? NG * kTile * 4 : 0;
    constexpr int kVBuf = kVBytes + kSBytes + 2 * kTile * 4;      // behind V: K scales of 8-bit codes, a wild tile's units
    constexpr int kMain = 2 * kKBytes + 3 * kVBuf;
    constexpr bool kLo = ROT;                          // the queries' second parts stay in LDS: a lane's own fragments
    __shared__ __align__(16) uint8_t lds[kMain + (kLo ? NW * NK * 1024 : 0)];
    uint8_t *const qlo = lds + kMain + (threadIdx.x >> 6) * (NK * 1024) + (threadIdx.x & 63) * 16;
    __shared__ int reach_all[NW][3];
    // what the columns see, read back only for tiles that need masks or distances
    __shared__ __align__(16) uint8_t cols[NW * 32 * sizeof(Column)];
    typedef TileRegs<D, BITS, NT> Regs;
    constexpr int UPT = Regs::UPT, KU = Regs::kU, FS = Regs::FS;

    const AttnTile id = attn_tile(a, ctiles);
    if (!id.valid) return;
    const int b = id.b, h = id.h, ct = id.ct, split = id.split;
    int s0;
    const int nall = ragged_rows(a.starts, b, a.total, &s0), n = min(nall, a.max_q), ncol = n * a.G;
    if (ct * 32 * NW >= ncol) return;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, m = lane & 31, hh = lane >> 5;
    const int len = cache_len(a.c, b), base = a.c.lens[b] - nall;
    const int prefix = a.prefix ? a.prefix[b] : 0;
    const int c0 = (ct * NW + wave) * 32;              // this wave's columns
    const bool active = c0 < ncol;

    // token (feature) of row m of a product: bits 2 and 3 exchanged, so that a lane's
    // results j = 8 t + i are tokens (features) 16 t + 8 hh + i: two operands of a
    // following product, or two pieces of 8 in memory
    const int mtok = (m & 19) | ((m & 4) << 1) | ((m & 8) >> 1);

    // ---- the query rows' loads, on the way while the columns and the first tile are
    // found: lane (column m, half hh) has features 16 k + 8 hh + e of its row
    uint4 qraw[NK];
    {
        const int c = c0 + m, cq = c < ncol ? c : c0 < ncol ? ncol - 1 : 0;      // (a column past the last repeats one)
        const uint16_t *row = static_cast<const uint16_t *>(a.q.ptr) + (int64_t)(s0 + cq / a.G) * a.q.ts +
                              (h * a.G + cq % a.G) * a.q.hs + 8 * hh;
#pragma unroll
        for (int k = 0; k < NK; ++k) qraw[k] = *reinterpret_cast<const uint4 *>(row + 16 * k);
    }

    // ---- what the wave's columns see, and the workgroup's range of tiles
    const int c = c0 + m;
    const bool cv = c < ncol;
    const Column mine(a, s0, n, base, len, prefix, h, c, cv);
    if (hh == 0) reinterpret_cast<Column *>(cols)[32 * wave + m] = mine;
    auto column = [&]() -> const Column & { return reinterpret_cast<const Column *>(cols)[32 * wave + m]; };
    Reach reach(mine, cv);
    reach.join<32>();
    reach.clip(a, len, prefix);
    reach.uniform();
    if (lane == 0) {
        reach_all[wave][0] = active ? reach.begin(prefix) : 0x7FFFFFFF;
        reach_all[wave][1] = active ? reach.hi_any : 0;
        reach_all[wave][2] = active ? reach.lo_any : 0x7FFFFFFF;
    }
    __syncthreads();
    int begin = 0x7FFFFFFF, end = 0, lo_any = 0x7FFFFFFF;
#pragma unroll
    for (int x = 0; x < NW; ++x) {
        begin = min(begin, reach_all[x][0]);
        end = max(end, reach_all[x][1]);
        lo_any = min(lo_any, reach_all[x][2]);
    }
    begin = __builtin_amdgcn_readfirstlane(begin);
    end = __builtin_amdgcn_readfirstlane(end);
    lo_any = __builtin_amdgcn_readfirstlane(lo_any);
    const int tile0 = begin / kTile, ntile = end > begin ? (end + kTile - 1) / kTile - tile0 : 0;
    const int per = max((ntile + a.splits - 1) / a.splits, a.least / kTile);
    const int ts = tile0 + split * per, te = min(ts + per, tile0 + ntile);

    const int P = 1 << a.c.page_shift;
    const PageLayout pl = page_layout(P, D, BITS);
    // ---- queries, divided by a power of two, in fp16
    f16x8 qf[NK];
    float qmul = 0.f;                                  // what the column's scores are multiplied with
    auto queries = [&]() {
        float x[NF][16];                               // features 32 i + 16 t + 8 hh + e at [i][8 t + e]
        uint4 (&q)[NK] = qraw;
        if constexpr (ROT) {
            // H (s o q) as a product with the +-1 matrix: exact bf16 operands, fp32 sums
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                const uint32_t sb = sign_byte(a.c.sk, 2 * k + hh);
                q[k].x ^= sign_pair(sb, 0);
                q[k].y ^= sign_pair(sb, 2);
                q[k].z ^= sign_pair(sb, 4);
                q[k].w ^= sign_pair(sb, 6);
            }
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const uint32_t f = 32 * i + mtok;
                f32x16 y{};
                uint32_t b[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) b[r] = sign_ones(f, 2 * r);
#pragma unroll
                for (int k = 0; k < NK; ++k)
                    y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(sign_frag(b, f, 16 * k + 8 * hh), __builtin_bit_cast(bf16x8, q[k]), y, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[i][e] = y[e];
            }
        } else {
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[k / 2][8 * (k & 1) + e] = __uint_as_float((e & 1) ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16));
            }
        }
        // 2^-ex brings the row's largest feature to [1, 2); its inverse goes into qmul
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[i][e]));
        top = fmaxf(top, __shfl_xor(top, 32));
        const int ex = min(max((int)(__float_as_uint(top) >> 23), 1), 253);
        const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
        qmul = __uint_as_float((uint32_t)ex << 23) * (!ROT ? 1.f : D == 128 ? 0.08838834764831845f : 0.125f);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x0 = x[k / 2][8 * (k & 1) + 2 * i] * down, x1 = x[k / 2][8 * (k & 1) + 2 * i + 1] * down;
                hi[i] = f16_pair(x0, x1);
                if constexpr (kLo) lo[i] = f16_pair(x0 - (float)h2(hi[i])[0], x1 - (float)h2(hi[i])[1]);
            }
            qf[k] = __builtin_bit_cast(f16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            if constexpr (kLo) *reinterpret_cast<uint4 *>(qlo + k * 1024) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    };
    f32x16 acc[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) acc[i] = f32x16{};
    float mrun = neg_inf(), lrun = 0.f;
    int erun = kTop;                                   // exponent field of acc's unit, by column
    float mul = 0.f;                                   // by column: log2 e times the scale
    const bool capped = a.cap > 0.f, sloped = a.slopes != nullptr, tree = a.tree != nullptr;

    // tiles between a prefix and the window are skipped by the whole workgroup
    auto next_tile = [&](int t) {
        const int skip_to = lo_any / kTile;
        return t * kTile >= prefix && t < skip_to ? skip_to : t;
    };
    // Pages of the tiles' halves, 32 tiles' worth in a register (lane 2 i + half:
    // tile seen + i) and loaded anew when a tile lies past them, so that the tile
    // loop holds no scalar load (it would drain with the LDS reads).
    int seen = ts, pages;
    auto load_pages = [&]() {
        const int tok = (seen + (lane >> 1)) * kTile + 32 * (lane & 1);
        pages = tok < len && seen + (lane >> 1) < te ? cache_page(a.c, b, tok) : -1;
    };
    auto page_of = [&](int t, int half) -> int { return __builtin_amdgcn_readlane(pages, 2 * (t - seen) + half); };
    // units of K: consecutive ones of a row; units of V: features f, f + FS, .. of
    // a block of 8 tokens.  The first half of the waves has the tile's first 32
    // tokens, so that a wave reads one page.
    const int kidx = tid * UPT, ktok = kidx / (D / 8), ku0 = kidx % (D / 8);
    const int vblk = tid / FS, vf = tid % FS;
    const bool second = __builtin_amdgcn_readfirstlane(wave) >= NW / 2;
    const uint32_t koff = (ktok & 31) * (D * BITS / 8) + ku0 * (4 * KU), voff = (vblk & 3) * (D * BITS) + vf * (4 * KU);
    const uint32_t all_off = (uint32_t)(hh ? pl.v_scales : pl.k_scales) + ((NG == 2 ? m >> 4 : 0) * P + 2 * (m & 15)) * 2;
    Regs rg, rg2;                                      // (rg2: the first tile)
    // The loads go through buffer descriptors of the two page blocks: a uniform
    // base, a uniform offset and one 32-bit offset a lane, bounded by the block.
    auto block = [&](int page) {
        // a half without a page reads page 0 (never used: its scales count as 0)
        const uint8_t *p = a.c.pool + (page >= 0 ? cache_block_offset(a.c, page, h) : 0);
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, (int)pl.bytes, 0x00027000);
    };
    auto r0 = block(-1), r1 = r0;                      // the tile's halves
    constexpr int kFetch = 4;                          // parts of a fetch
    auto fetch_part = [&](Regs &rg, int part, int t, int p0, int p1) {
        const int t0 = t * kTile, i0 = t0 & (P - 1), i1 = (t0 + 32) & (P - 1), iw = second ? i1 : i0;
        if (part == 0) {
            r0 = block(p0);
            r1 = block(p1);
        }
        const auto bw = second ? r1 : r0;
        if (part == 1) {
            constexpr int N = UPT * KU;
            if constexpr (N == 1) rg.k[0] = __builtin_amdgcn_raw_buffer_load_b32(bw, koff, iw * (D * BITS / 8), 0);
            else if constexpr (N == 2) {
                const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(bw, koff, iw * (D * BITS / 8), 0);
                rg.k[0] = v.x; rg.k[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(bw, koff + 4 * i, iw * (D * BITS / 8), 0);
                    rg.k[i] = v.x; rg.k[i + 1] = v.y; rg.k[i + 2] = v.z; rg.k[i + 3] = v.w;
                }
            }
#pragma unroll
            for (int q = 0; q < NG; ++q)
                rg.ks[q] = __builtin_amdgcn_raw_buffer_load_b16(bw, (ktok & 31) * 2, (int)pl.k_scales + (q * P + iw) * 2, 0);
        }
        if (part == 2) {
#pragma unroll
            for (int x = 0; x < UPT; ++x) {
                const int so = (int)pl.v_codes + (iw >> 3) * (D * BITS);
                if constexpr (KU == 1) rg.v[x] = __builtin_amdgcn_raw_buffer_load_b32(bw, voff + FS * x * 4, so, 0);
                else {
                    const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(bw, voff + FS * x * 8, so, 0);
                    rg.v[2 * x] = v.x; rg.v[2 * x + 1] = v.y;
                }
            }
        }
        if (part == 3) {
#pragma unroll
            for (int q = 0; q < NG; ++q) {
                const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(bw, (vblk & 3) * 16, (int)pl.v_scales + (q * P + iw) * 2, 0);
                rg.vs[q][0] = v.x; rg.vs[q][1] = v.y; rg.vs[q][2] = v.z; rg.vs[q][3] = v.w;
            }
            rg.all[0] = __builtin_amdgcn_raw_buffer_load_b32(r0, all_off, i0 * 2, 0);
            rg.all[1] = __builtin_amdgcn_raw_buffer_load_b32(r1, all_off, i1 * 2, 0);
        }
    };
    auto fetch = [&](Regs &rg, int t, int p0, int p1) {
#pragma unroll
        for (int x = 0; x < kFetch; ++x) fetch_part(rg, x, t, p0, p1);
    };
    // Of the scales of K (lane 31) and of V (lane 63): the largest in the lower half,
    // the smallest that is not 0 in the upper one, negated, so that one maximum over
    // rows of 16 and then the second row of each half finds both.
    auto extremes = [&](uint32_t a0, uint32_t a1) {
        const u16x2 z{0, 0}, b0 = __builtin_bit_cast(u16x2, a0), b1 = __builtin_bit_cast(u16x2, a1);
        const uint32_t x = pk_umax(a0, a1), y = pk_umax(__builtin_bit_cast(uint32_t, (u16x2)(z - b0)), __builtin_bit_cast(uint32_t, (u16x2)(z - b1)));
        uint32_t v = pk_umax(__builtin_amdgcn_perm(y, x, 0x05040100u), __builtin_amdgcn_perm(y, x, 0x07060302u));
        v = pk_umax(v, dpp_u<kDppXor1>(v));
        v = pk_umax(v, dpp_u<kDppXor2>(v));
        v = pk_umax(v, dpp_u<kDppHalfMirror>(v));
        v = pk_umax(v, dpp_u<kDppMirror>(v));
        return pk_umax(v, dpp_u<kDppRowBcast15>(v));
    };
    auto lane_of = [](uint32_t v, int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); };
    // registers -> LDS.  Sets the tile's K and V units (exponent fields) and whether
    // its scales spread too far for one unit (wild: every token then has its own).
    int vunit_now = 0;                                 // V unit of the last tile, 0: none yet
    uint32_t magic = 0x64006400u;
    asm("" : "+v"(magic));
    struct Tile { int t, p0, p1, ek, ev, wild; };
    uint32_t kbad = 0, kdown = 0, vdown[4];
    auto units = [&](Regs &rg, Tile &tile, uint8_t *vbuf) {
        const int t0 = tile.t * kTile;
        const int lim0 = tile.p0 >= 0 ? len : 0, lim1 = tile.p1 >= 0 ? len : 0;      // tokens below these count, by half
        const bool whole = t0 + kTile <= min(lim0, lim1);
        uint32_t all0 = rg.all[0], all1 = rg.all[1];
        if (!whole) {
            const int ta = t0 + 2 * (m & 15), tb = ta + 32;
            all0 &= (ta < lim0 ? 0xFFFFu : 0u) | (ta + 1 < lim0 ? 0xFFFF0000u : 0u);
            all1 &= (tb < lim1 ? 0xFFFFu : 0u) | (tb + 1 < lim1 ? 0xFFFF0000u : 0u);
        }
        uint32_t x = extremes(all0, all1);
        uint32_t xk = lane_of(x, 31), xv = lane_of(x, 63);
        const bool clean = whole && max(xk & 0xFFFFu, xv & 0xFFFFu) < 0x7F80u;
        kbad = 0;
        const int limw = second ? lim1 : lim0, tk = t0 + ktok, tv = t0 + 8 * vblk;
        if (!clean) {
            // a tile with a last token, a missing half or a NaN scale inside: scales
            // that do not count become 0, and a NaN of K or V goes into the K row
            auto finite = [&](uint32_t two, int tt, int lim) -> uint32_t {
                if (tt >= lim || (two & 0x7F80u) == 0x7F80u) two &= 0xFFFF0000u;
                if (tt + 1 >= lim || (two & 0x7F800000u) == 0x7F800000u) two &= 0x0000FFFFu;
                return two;
            };
            all0 = finite(all0, 0, 2);
            all1 = finite(all1, 0, 2);
            x = extremes(all0, all1);
            xk = lane_of(x, 31);
            xv = lane_of(x, 63);
            const int pw = second ? tile.p1 : tile.p0;
            if (tk < limw) {                           // limw > 0: the half has a page
                const uint8_t *sv = a.c.pool + cache_block_offset(a.c, max(pw, 0), h) + pl.v_scales;
                const uint32_t vs0 = reinterpret_cast<const uint16_t *>(sv)[tk & (P - 1)];
                if ((rg.ks[0] & 0x7F80u) == 0x7F80u || (vs0 & 0x7F80u) == 0x7F80u) kbad = 0x7E007E00u;
            } else {
#pragma unroll
                for (int q = 0; q < NG; ++q) rg.ks[q] = 0;
            }
#pragma unroll
            for (int q = 0; q < NG; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) rg.vs[q][i] = finite(rg.vs[q][i], tv + 2 * i, limw);
        }
        // exponents of the largest scales and of the smallest (none: 512)
        const uint32_t zv = xv & 0xFFFFu;
        const int ek = max((int)((xk & 0xFFFFu) >> 7), kTop), ev = max((int)(zv >> 7), kTop);
        const int lk = (int)((0x10000u - (xk >> 16)) >> 7), lv = (int)((0x10000u - (xv >> 16)) >> 7);
        // V keeps its unit from tile to tile while the largest scale is at most 2^8
        // below it, and raises it by up to 2^4; scales more than 2^18 below count fully
        // only where every token has its own unit
        const bool jump = vunit_now != 0 && (ev > vunit_now + 4 || ev < vunit_now - 8) && zv != 0;
        if (zv != 0) vunit_now = jump || vunit_now == 0 ? ev : max(vunit_now, ev);
        const int vu = max(vunit_now, kTop);
        tile.wild = jump || (!kPost && lk < ek - 18) || lv < vu - 18;
        tile.ek = ek;
        tile.ev = tile.wild ? ev : vu;
        kdown = (uint32_t)(ek - kTop) * 0x00800080u;
#pragma unroll
        for (int i = 0; i < 4; ++i) vdown[i] = (uint32_t)(vu - kTop) * 0x00800080u;
        if (tile.wild) {
            float *km = reinterpret_cast<float *>(vbuf + kVBytes + kSBytes);
            int *ve = reinterpret_cast<int *>(km + kTile);
            const int e = max((int)(max((uint32_t)rg.ks[0], (uint32_t)rg.ks[NG - 1]) >> 7), kTop);
            const int ec = kbad ? kTop : e;            // (a NaN scale's exponent is no unit)
            kdown = (uint32_t)(ec - kTop) * 0x00800080u;
            if (ku0 == 0) km[ktok] = __builtin_ldexpf(1.f, ec - 127 - (kTop - 15));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t two = NG == 1 ? rg.vs[0][i] : pk_umax(rg.vs[0][i], rg.vs[NG - 1][i]);
                const int e0 = max((int)((two >> 7) & 255u), kTop), e1 = max((int)(two >> 23), kTop);
                vdown[i] = (uint32_t)(e0 - kTop) * 0x80u + (uint32_t)(e1 - kTop) * 0x00800000u;
                if (vf == 0) {
                    ve[8 * vblk + 2 * i] = e0;
                    ve[8 * vblk + 2 * i + 1] = e1;
                }
            }
        }
    };
    // registers -> LDS, in 2 UPT parts: the thread's units of K, then those of V
    auto put = [&](const Regs &rg, int part, uint8_t *kbuf, uint8_t *vbuf) {
        if (part < UPT) {
            const int x = part, u = ku0 + x, g = u / (D / 32), kk = u % (D / 32);
            f16x2 y[4];
            unit_f16<BITS>(&rg.k[x * KU], magic, y);
            if constexpr (!kPost) {
                // kk runs from ku0 % (D/32) on: with D / 32 <= 4 its group is known or one of two
                const uint32_t s = NG == 1 ? rg.ks[0] : (kk & 2 ? rg.ks[NG - 1] : rg.ks[0]);
                const f16x2 sc = h2(u32(scale_f16(s | (s << 16), kdown)) | kbad);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] *= sc;
            }
            *reinterpret_cast<uint4 *>(kbuf + (4 * kk + g) * kKStride + ktok * 16) =
                make_uint4(u32(y[0]), u32(y[1]), u32(y[2]), u32(y[3]));
            if constexpr (kPost) {
                if (part == 0 && ku0 == 0)
#pragma unroll
                    for (int q = 0; q < NG; ++q)
                        reinterpret_cast<float *>(vbuf + kVBytes)[q * kTile + ktok] =
                            kbad ? __builtin_nanf("") : bf16_to_f32(rg.ks[q]);
            }
        } else {
            const int x = part - UPT, q = NG == 1 ? 0 : (FS * x) / 64;
            f16x2 y[4];
            unit_f16<BITS>(&rg.v[x * KU], magic, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] *= scale_f16(rg.vs[q][i], vdown[i]);
            *reinterpret_cast<uint4 *>(vbuf + (vblk * D + vf + FS * x) * 16) =
                make_uint4(u32(y[0]), u32(y[1]), u32(y[2]), u32(y[3]));
        }
    };

    uint8_t *const vlds = lds + 2 * kKBytes;

    // Two groups of waves, one on each half of every SIMD's slots, take turns at
    // the matrix cores: while one multiplies (weights of its last tile times V,
    // then queries times the K of the next) and writes its half of the tile after
    // to LDS in between, the other runs softmax on the vector unit and finds the
    // units of the tile after that; a barrier ends each turn.
    //   turn    2 i           2 i + 1        2 i + 2        2 i + 3
    //   early   M(i) put i+1  V(i) units i+2 M(i+1) put i+2 V(i+1)
    //   late    V(i-1)        M(i) put i+1   V(i) units i+2 M(i+1) put i+2
    // M(i) multiplies with V(i-1) and K(i).  Tile i + 1 is whole before turn 2 i + 2,
    // and is put in turns 2 i and 2 i + 1 where K(i), V(i-1) are read and, by then
    // done with, K(i-1) and V(i-2) were: two K buffers, three V buffers.
    const bool late = second;
    auto look = [&](int t) {
        if (t >= te) return Tile{t, -1, -1, kTop, kTop, 0};
        if (t >= seen + 32) {
            seen = t;
            load_pages();
        }
        return Tile{t, page_of(t, 0), page_of(t, 1), kTop, kTop, 0};
    };
    auto kbuf_of = [&](int nth) { return lds + (nth & 1) * kKBytes; };
    auto vbuf_of = [&](int nth) { return vlds + (nth % 3) * kVBuf; };
    f32x16 s[2];
    f16x8 pf[4];
    // In both products the next step's fragments are read from LDS before the
    // present step's products are issued, in the order written here.
    auto times_v = [&](int nth) {
        const uint8_t *vb = vbuf_of(nth);
        uint8_t *const kput = kbuf_of(nth + 2), *const vput = vbuf_of(nth + 2);
        constexpr int A = 5;                           // pairs of fragments held: four ahead of the one in use
        f16x8 f[A][2];
        auto read = [&](int g) {                       // pair g: block of tokens g / (NF/2), features of 2 (g % (NF/2))
#pragma unroll
            for (int i = 0; i < 2; ++i)
                f[g % A][i] = *reinterpret_cast<const f16x8 *>(
                    vb + ((2 * (g / (NF / 2)) + hh) * D + 32 * (2 * (g % (NF / 2)) + i) + m) * 16);
        };
        constexpr int N = 4 * NF / 2;
        static_assert(N == 4 * UPT);
#pragma unroll
        for (int g = 0; g < A - 1; ++g) read(g);
#pragma unroll
        for (int g = 0; g < N; ++g) {
            if (g + A - 1 < N) read(g + A - 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = 2 * (g % (NF / 2)) + i;
                acc[x] = mfma32(f[g % A][i], pf[g / (NF / 2)], acc[x]);
            }
            if (g & 1) put(rg, g >> 1, kput, vput);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // between: what else is issued after step k's products
    auto times_k = [&](int nth, auto between) {
        const uint8_t *kb = lds + (nth & 1) * kKBytes;
        // x[u] += K rows of half u times the queries, features 16 k0 .. 16 k1 - 1
        auto products = [&](f32x16 (&x)[2], int k0, int k1) {
            constexpr int A = kPost ? 2 : 3;           // steps held: the ones ahead of the one in use
            f16x8 kf[A][2], ql[A];
            auto read = [&](int k) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    kf[k % A][u] = *reinterpret_cast<const f16x8 *>(kb + (2 * k + hh) * kKStride + (32 * u + mtok) * 16);
                if constexpr (kLo) ql[k % A] = *reinterpret_cast<const f16x8 *>(qlo + k * 1024);
            };
#pragma unroll
            for (int k = k0; k < k0 + A - 1; ++k) read(k);
#pragma unroll
            for (int k = k0; k < k1; ++k) {
                if (k + A - 1 < k1) read(k + A - 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int u = 0; u < 2; ++u) x[u] = mfma32(kf[k % A][u], qf[k], x[u]);
                if constexpr (kLo)
#pragma unroll
                    for (int u = 0; u < 2; ++u) x[u] = mfma32(kf[k % A][u], ql[k % A], x[u]);
                between(k);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if constexpr (kPost) {
            const float *ks = reinterpret_cast<const float *>(vlds + (nth % 3) * kVBuf + kVBytes) + 8 * hh;
#pragma unroll
            for (int q = 0; q < NG; ++q) {
                f32x16 x[2] = {f32x16{}, f32x16{}};
                products(x, 4 * q, 4 * q + 4);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(ks + q * kTile + 32 * u + (e >> 3) * 16 + (e & 7));
                        const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            s[u][e + y] = q == 0 ? x[u][e + y] * ff[y] : fmaf(x[u][e + y], ff[y], s[u][e + y]);
                    }
            }
        } else {
            s[0] = s[1] = f32x16{};
            products(s, 0, NK);
        }
    };

    const int first_tile = next_tile(ts);
    if (a.c.pages > 0 && first_tile < te) {            // (no page: nothing to see)
        seen = first_tile;
        load_pages();
        Tile cur = look(first_tile), nxt = look(next_tile(first_tile + 1));
        fetch(rg2, cur.t, cur.p0, cur.p1);
        fetch(rg, nxt.t, nxt.p0, nxt.p1);
        queries();
        mul = fminf(a.scale * kLog2e * qmul, 3e38f);   // (finite: a score of 0 stays 0)
        units(rg2, cur, vbuf_of(0));
#pragma unroll
        for (int x = 0; x < 2 * UPT; ++x) put(rg2, x, kbuf_of(0), vbuf_of(0));
        units(rg, nxt, vbuf_of(1));
        Tile nx2 = look(next_tile(nxt.t + 1));
        __syncthreads();
        if (late) __syncthreads();                     // the late group's first turn: early multiplies
#pragma unroll
        for (int x = 0; x < 2 * UPT; ++x) put(rg, x, kbuf_of(1), vbuf_of(1));
        fetch(rg, nx2.t, nx2.p0, nx2.p1);
        times_k(0, [](int) {});
        erun = cur.ev;
        __syncthreads();
        for (int i = 0;; ++i) {
            const int t0 = cur.t * kTile;
            const Tile nx3 = look(next_tile(nx2.t + 1));
            // ---- V: softmax of this tile, units of a later one
            const float *km = reinterpret_cast<const float *>(vlds + (i % 3) * kVBuf + kVBytes + kSBytes) + 8 * hh;
            float kunit = kPost ? 1.f : __builtin_ldexpf(1.f, cur.ek - 127 - (kTop - 15));   // 2^E
            if (!kPost && cur.wild) {                  // a unit for every token
                kunit = 1.f;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[u][e] *= km[32 * u + (e >> 3) * 16 + (e & 7)];
            }
            // scores in units of `unit` (log2 e times the scale's factors; not so small that
            // a masked score's -inf would meet a 0), or, where the terms are not linear, in
            // log2 units already
            float unit = fmaxf(mul * kunit, 1e-30f);
            if (capped) {
                const float scap = fminf(a.scale / a.cap * (2.f * kLog2e) * qmul * kunit, 3e38f);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float x = __builtin_amdgcn_exp2f(-fabsf(s[u][e] * scap));
                        s[u][e] = copysignf((1.f - x) * __builtin_amdgcn_rcpf(1.f + x), s[u][e]) * (a.cap * kLog2e);
                    }
                unit = 1.f;
            }
            if (sloped) {
                const Column col = column();
                const bool slots = tree && t0 + kTile > base;
                const float far = (float)(col.pos - t0 - 8 * hh);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int t = 32 * u + (e >> 3) * 16 + (e & 7);
                        float dist = fabsf(far - (float)t);
                        if (slots) dist = col.distance(a, t0 + 8 * hh + t, s0, n, base);
                        s[u][e] = fmaf(s[u][e], unit, -col.slope * dist);
                    }
                unit = 1.f;
            }
            const bool full = cur.p0 >= 0 && cur.p1 >= 0 && t0 >= reach.lo_all && t0 + kTile <= reach.hi_all;
            if (!full) {
                const Column col = column();
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t vis = col.sees8(tree, base, t0 + 32 * u + 16 * x + 8 * hh);
                        if ((u ? cur.p1 : cur.p0) < 0) vis = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {         // all ones or zeros from the bit picks the score or -inf
                            const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)vis, e, 1);
                            s[u][8 * x + e] = __uint_as_float((__float_as_uint(s[u][8 * x + e]) & keep) | (~keep & 0xFF800000u));
                        }
                    }
            }
            float mx = s[0][0];
#pragma unroll
            for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s[0][e]);
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[1][e]);
            mx *= unit;
            if (__any(mx > mrun + 8.f)) {
                mx = fmaxf(fmaxf(mx, __shfl_xor(mx, 32)), mrun);
                const float alpha = mx == mrun ? 1.f : __builtin_amdgcn_exp2f(mrun - mx);
                mrun = mx;
                lrun *= alpha;
#pragma unroll
                for (int x = 0; x < NF; ++x) acc[x] *= alpha;
            }
            float mu = mrun == neg_inf() ? 0.f : -mrun, lsum = 0.f;
            const bool shift = cur.wild || __any(erun != cur.ev);
            if (shift || __any(fabsf(mu) > 1e6f)) {
                // scores so large that their own rounding counts, and weights in another
                // unit, take the difference to the maximum here
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[u][e] = s[u][e] * unit + mu;
                unit = 1.f;
                mu = 0.f;
                if (shift) {
                    // Another unit of V.  A column takes the tile's, unless its sum would leave
                    // 2^-40 .. 2^100 there or every token has its own: then the one in which its
                    // largest weight is 1 to 2, or its sum at 2^100 if that is larger (what the
                    // other side then loses is below 2^-60 of the whole).
                    float top = neg_inf(), atop = 0.f;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 16; ++e) lsum += __builtin_amdgcn_exp2f(s[u][e]);
                    if (cur.wild) {
                        const int *ve = reinterpret_cast<const int *>(km + kTile);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int e = 0; e < 16; ++e) s[u][e] += (float)(ve[32 * u + (e >> 3) * 16 + (e & 7)] - cur.ev);
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[u][e]);
#pragma unroll
                    for (int x = 0; x < NF; ++x)
#pragma unroll
                        for (int e = 0; e < 16; ++e) atop = fmaxf(atop, fabsf(acc[x][e]));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    atop = fmaxf(atop, __shfl_xor(atop, 32));
                    constexpr int kNone = -4096;
                    const int we = top > -1000.f ? cur.ev + (int)floorf(top) : kNone;
                    const int ae = atop > 0.f ? erun + (int)(__float_as_uint(atop) >> 23) - 127 : kNone;
                    int en = max(we, ae - 100);
                    if (en <= kNone || (!cur.wild && (ae == kNone || (ae >= cur.ev - 40 && ae <= cur.ev + 100)))) en = cur.ev;
#pragma unroll
                    for (int x = 0; x < NF; ++x)
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[x][e] = __builtin_ldexpf(acc[x][e], erun - en);
                    mu = (float)(cur.ev - en);
                    erun = en;
                    lsum += lrun;
                }
                asm("" : "+v"(s[0]), "+v"(s[1]));      // in place: no copies on the way past
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    s[u][e] = __builtin_amdgcn_exp2f(fmaf(s[u][e], unit, mu));
                    lrun += s[u][e];
                }
            if (shift) lrun = lsum;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const f32x16 &p = s[x >> 1];
                const int o = 8 * (x & 1);
                pf[x] = __builtin_bit_cast(f16x8, make_uint4(f16_pair(p[o], p[o + 1]), f16_pair(p[o + 2], p[o + 3]),
                                                             f16_pair(p[o + 4], p[o + 5]), f16_pair(p[o + 6], p[o + 7])));
                asm volatile("" : "+v"(pf[x]), "+v"(lrun));   // computed in this turn, not sunk into the next
            }
            units(rg, nx2, vbuf_of(i + 2));
            __syncthreads();
            // ---- M: products, and tile i + 2 to LDS
            const bool last = nxt.t >= te;
            __builtin_amdgcn_s_setprio(1);             // before the other group's vector work: 434 -> 415 us
            times_v(i);
            if (last) break;
            times_k(i + 1, [&](int k) {
                if (k % (NK / kFetch) == 0) fetch_part(rg, k / (NK / kFetch), nx3.t, nx3.p0, nx3.p1);
            });
            __builtin_amdgcn_s_setprio(0);
            __syncthreads();
            cur = nxt;
            nxt = nx2;
            nx2 = nx3;
        }
        if (!late) __syncthreads();
    }
    __syncthreads();

    // ---- rows out: lane (column m, half hh) has features 32 i + 8 (j / 4) + 4 hh + j % 4
    if (!active) return;
    lrun += __shfl_xor(lrun, 32);
    mrun = nan_outweighs(mrun, lrun);
    const int vexp = erun - 127 - (kTop - 15);
    const int64_t qrow = s0 + (cv ? c / a.G : 0);
    const int head = h * a.G + (cv ? c % a.G : 0);
    if (a.splits > 1) {
        if (!cv) return;
        const int64_t rows = (int64_t)a.total * a.hq, at = split * rows + qrow * a.hq + head;
        if (hh == 0) {
            a.ws_ml[2 * at] = mrun;
            a.ws_ml[2 * at + 1] = lrun;
        }
        if (mrun == neg_inf()) return;
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *reinterpret_cast<float4 *>(a.ws_part + at * D + 32 * i + 8 * y + 4 * hh) =
                    make_float4(__builtin_ldexpf(acc[i][4 * y], vexp), __builtin_ldexpf(acc[i][4 * y + 1], vexp),
                                __builtin_ldexpf(acc[i][4 * y + 2], vexp), __builtin_ldexpf(acc[i][4 * y + 3], vexp));
        return;
    }
    const float inv = lrun == 0.f ? 0.f : 1.f / lrun;
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = __builtin_ldexpf(acc[i][e] * inv, vexp);
    const RowEnd fin = cv ? row_end(a, qrow * a.hq + head, mrun, lrun) : RowEnd{0.f, 0.f, 0.f};
    if (cv && a.lse && hh == 0) a.lse[qrow * a.hq + head] = fin.lse;
    if constexpr (ROT) {
        // back through H: the sums in two bf16 parts (2^-16 of the row's largest) times
        // +-1; element e of step t is feature 16 t + 8 (e / 4) + 4 hh + e % 4
        bf16x8 hi[NK], lo[NK];
#pragma unroll
        for (int t = 0; t < NK; ++t) {
            uint32_t u[4], v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float x0 = acc[t / 2][8 * (t & 1) + 2 * r], x1 = acc[t / 2][8 * (t & 1) + 2 * r + 1];
                u[r] = bf16_pair(x0, x1);
                v[r] = bf16_pair(x0 - __uint_as_float(u[r] << 16), x1 - __uint_as_float(u[r] & 0xFFFF0000u));
            }
            hi[t] = __builtin_bit_cast(bf16x8, make_uint4(u[0], u[1], u[2], u[3]));
            lo[t] = __builtin_bit_cast(bf16x8, make_uint4(v[0], v[1], v[2], v[3]));
        }
        const float isd = D == 128 ? 0.08838834764831845f : 0.125f;
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            const uint32_t f = 32 * i + mtok;
            const uint32_t b[4] = {sign_ones(f, 0), sign_ones(f, 2), sign_ones(f, 8), sign_ones(f, 10)};
            f32x16 y{};
#pragma unroll
            for (int t = 0; t < NK; ++t) {
                const bf16x8 hf = sign_frag(b, f, 16 * t + 4 * hh);
                y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hf, hi[t], y, 0, 0, 0);
                y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hf, lo[t], y, 0, 0, 0);
            }
            if (cv)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t sb = sign_byte(a.c.sv, 4 * i + 2 * t + hh);
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = flip(y[8 * t + e] * isd, (sb >> e) & 1);
                    store_out8<D>(a, qrow, head, 32 * i + 16 * t + 8 * hh, o, fin);
                }
        }
    } else {
        // pieces of 4 features: this lane's and those of its neighbour half make pieces of 8
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                // registers 8 t + 0..3: features 16 t + 4 hh ..; 8 t + 4..7: 16 t + 8 + 4 hh ..
                float o[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a0 = acc[i][8 * t + e], a1 = acc[i][8 * t + 4 + e];
                    const float other = __shfl_xor(hh ? a0 : a1, 32);
                    o[e] = hh ? other : a0;
                    o[4 + e] = hh ? a1 : other;
                }
                if (cv) store_out8<D>(a, qrow, head, 32 * i + 16 * t + 8 * hh, o, fin);
            }
    }
}

template <int D, int BITS, bool ROT>
static hipError_t wide_launch(const CacheAttnArgs &a, hipStream_t s) {
    constexpr int NW = 8;
    const int64_t ctiles = ((int64_t)a.max_q * a.G + 32 * NW - 1) / (32 * NW);
    const int64_t grid = attn_grid((int64_t)a.c.batch * a.c.H, a.splits * ctiles);
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    KTimeScope kts("k_cache_attn_wide", s);
    hipLaunchKernelGGL((k_cache_attn_wide<D, BITS, ROT, NW>), dim3((unsigned)grid), dim3(64 * NW), 0, s, a, (int)ctiles);
    return hipGetLastError();
}
template <int D>
static hipError_t wide_d(const CacheAttnArgs &a, int bits, bool rotate, hipStream_t s) {
    if (bits == 4) return rotate ? wide_launch<D, 4, true>(a, s) : wide_launch<D, 4, false>(a, s);
    return rotate ? wide_launch<D, 8, true>(a, s) : wide_launch<D, 8, false>(a, s);
}
hipError_t launch_cache_attn_wide(const CacheAttnArgs &a, int d, int bits, bool rotate, hipStream_t s) {
    return d == 128 ? wide_d<128>(a, bits, rotate, s) : wide_d<64>(a, bits, rotate, s);
}

}  // namespace jolt
