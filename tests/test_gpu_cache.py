"""The token cache on the GPU against its oracle (oracle/cache.py).

Writing and keeping are compared byte for byte over the whole pool (the
rotation of bf16 rows is exact in fp64 and rounded once, so no code may differ;
bytes of other tokens must stay).

Reading: a value is isd (s0 I0 +- s1 I1), the I exact integers: one rounding of
2^-24 for each product, the sum and the scaling, and one in isd, all relative to
at most isd (|s0 I0| + |s1 I1|), then one to the output type (2^-24 or 2^-8).

Attention: the error of a score is at most
    delta = scale sum_f |q'_f| (2^-16 |k'_f| + 2^-24 (d + 4) (136 + 128) sc)
(rotated queries in two bf16 parts, 2^-8 of 2^-8, and fp32 sums of at most d
products of codes with their offset; unrotated queries are exact).  A weight
then errs by 2 delta relatively (numerator and denominator), by 2^-8 where it is
rounded to bf16 with its value scale, and by 2^-24 for each of the sum's
additions (at most T / 16 + 70 in a row) and 2^-20 for exponentials.  In norms,
which the rotation keeps: with A_f = sum_t p_t |v'_tf| in the stored domain,
    ||o - o_ref|| <= (2^-8 + 2 delta + tail) ||A|| + 2^-8 ||o_ref||
    |lse - lse_ref| <= delta + tail + 2^-20 (1 + |lse_ref|)
with tail = 2^-24 (T / 16 + 70) + 2^-20.
"""
import math

import numpy as np
import pytest

from oracle import attention as oatt, cache as oc
from tests.gpu_util import jolt_binding, torch_cuda

pytestmark = pytest.mark.gpu


def bf16(x):
    return oc.quant.round_bf16(x).astype(np.float32)


class Both:
    """One cache on the GPU and in the oracle, with the same pages and lengths."""

    def __init__(self, s, batch, max_pages, pages, seed=0, bad=()):
        self.torch, self.jb = torch_cuda(), jolt_binding()
        self.s, self.batch = s, batch
        r = np.random.default_rng(seed)
        pool = r.integers(0, 256, pages * s.H * s.head_bytes, dtype=np.uint8)     # leftovers, NaN scales among them
        table = np.full((batch, max_pages), -1, dtype=np.int32)
        ids = r.permutation(pages)
        for i in range(min(batch * max_pages, pages)):
            table[i // max_pages, i % max_pages] = ids[i]
        for b, p, x in bad:
            table[b, p] = x
        self.ref = oc.Cache(s, pool.copy(), table, [0] * batch)
        t = self.torch
        self.pool = t.from_numpy(pool).cuda()
        self.table = t.from_numpy(table).cuda()
        self.lens = t.zeros(batch, dtype=t.int32, device="cuda")
        self.gpu = self.jb.JoltCache(s.H, s.d, s.bits, self.pool, self.table, self.lens, page_tokens=s.P,
                                     rotate=s.rotate, seed=s.seed, k_item_id=s.k_id, v_item_id=s.v_id)

    def dev(self, x, dtype):
        t = self.torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
        return t if dtype == "f32" else t.bfloat16()

    def i32(self, x):
        return self.torch.tensor(list(x), dtype=self.torch.int32, device="cuda")

    def starts(self, n):
        return np.concatenate([[0], np.cumsum(n)]).astype(int)

    def set_lens(self, lens):
        self.ref.lens = list(lens)
        self.lens.copy_(self.i32(lens))

    def append(self, k, v, n, dtype="bf16", head_major=False):
        """k, v (total, H, d) fp32 (bf16-valued for bf16); lens set before."""
        st = self.starts(n)
        self.ref.append(k, v, st)
        d = [self.dev(x, dtype) for x in (k, v)]
        if head_major:
            d = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in d]
        self.gpu.append(d[0], d[1], self.i32(st), int(max(n)) if len(n) else 0)

    def grow(self, n, rng, dtype="bf16", **kw):
        self.set_lens([a + b for a, b in zip(self.ref.lens, n)])
        k, v = (rng.standard_normal((sum(n), self.s.H, self.s.d)).astype(np.float32) for _ in range(2))
        k[..., 3] *= 20.0
        if dtype == "bf16":
            k, v = bf16(k), bf16(v)
        self.append(k, v, n, dtype, **kw)
        return k, v

    def check_pool(self):
        got = self.pool.cpu().numpy().reshape(self.ref.pages.pool.shape)
        bad = np.argwhere(got != self.ref.pages.pool)
        assert len(bad) == 0, (len(bad), bad[:5])


SHAPES = [
    # H, d, bits, P, rotate
    (2, 128, 4, 64, True), (3, 128, 8, 32, True), (2, 128, 4, 256, False), (1, 128, 8, 128, False),
    (4, 64, 4, 32, True), (2, 64, 8, 64, True), (3, 64, 4, 64, False), (2, 64, 8, 32, False),
]
IDS = ["H%d_d%d_b%d_P%d_%s" % (h, d, b, p, "rot" if r else "plain") for h, d, b, p, r in SHAPES]


# ------------------------------------------------------------------ writing
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_append_bytes(shape, dtype):
    s = oc.Shape(*shape, seed=11, k_id=4, v_id=9)
    c = Both(s, 3, 3, 10, seed=1)
    rng = np.random.default_rng(5)
    for n in ([5, 1, 0], [1, 1, 1], [17, 2, 9], [0, 0, 31], [8, 8, 1], [1, 0, 1]):
        c.grow(n, rng, dtype, head_major=n[0] == 17)
        c.check_pool()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rotate", [False, True])
def test_append_extreme_rows(bits, rotate):
    s = oc.Shape(2, 128, bits, 32, rotate, seed=2)
    c = Both(s, 1, 2, 2)
    x = bf16(np.random.default_rng(3).standard_normal((12, 2, 128)))
    x[1] = 0
    x[2, 0, 70] = np.nan
    x[3, 1, 5] = -np.inf
    x[4] *= 1e-38
    x[5] *= 1e37
    x[6] = bf16(np.float32(3.0e38))
    x[7, :, :64] = 0
    x[8] = np.float32(2.0 ** -130)
    x[9, :, 0] = 1e20
    c.set_lens([12])
    c.append(x, x[::-1].copy(), [12], "f32")
    c.check_pool()


def test_append_left_out_tokens():
    """Pages outside the pool, tokens past the table or before 0, and rows past the last sequence."""
    s = oc.Shape(2, 64, 4, 32, True)
    c = Both(s, 4, 2, 9, bad=((0, 1, 9), (1, 0, -5)))
    rng = np.random.default_rng(0)
    n = [40, 50, 70, 6]
    c.set_lens([40, 50, 70, 2])               # 70 > 64 tokens of two pages; 2 < 6 rows
    k, v = (bf16(rng.standard_normal((sum(n) + 5, 2, 64))) for _ in range(2))
    c.append(k, v, n)
    c.check_pool()


def test_append_refuses_bad_offsets_quietly():
    """starts that run backwards or past the rows write nothing."""
    s = oc.Shape(1, 64, 8, 32, False)
    c = Both(s, 2, 1, 2)
    c.set_lens([8, 8])
    x = c.dev(np.ones((8, 1, 64)), "bf16")
    for st in ([0, -4, 8], [8, 4, 0], [5, 9, 12], [-2, 0, 0]):
        c.gpu.append(x, x, c.i32(st), 8)
        if st[1] < 0:
            continue
    c.torch.cuda.synchronize()
    c.check_pool()


# ------------------------------------------------------------------ reading
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_read_values(shape, dtype):
    s = oc.Shape(*shape, seed=5)
    c = Both(s, 3, 3, 10, seed=2)
    t = c.torch
    rng = np.random.default_rng(6)
    c.grow([37, 5, 1], rng)
    c.grow([20, 1, 0], rng)
    first, n = [3, 0, 0], [41, 6, 9]                                  # the last asks past its one token
    st = c.starts(n)
    total, spare = int(st[-1]), 4
    dt = t.float32 if dtype == "f32" else t.bfloat16
    out = [t.full((s.H, total + spare, s.d), 7.0, dtype=dt, device="cuda").transpose(0, 1) for _ in range(2)]
    c.gpu.read(c.i32(first), c.i32(st), max(n), out[0], out[1])
    got = [o.float().cpu().numpy().astype(np.float64) for o in out]
    isd = 1 / math.sqrt(s.d) if s.rotate else 1.0
    rnd = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    for b in range(3):
        for value, g in zip((False, True), got):
            want, _ = c.ref.rows(b, first[b], n[b], value)
            stored, _ = c.ref.rows(b, first[b], n[b], value, rotated=True)
            big = isd * np.abs(stored).sum(-1, keepdims=True) if s.rotate else np.abs(want)
            lim = 5 * 2.0 ** -24 * big + rnd * np.abs(want)
            assert np.all(np.abs(g[st[b]:st[b + 1]] - want) <= lim)
    for g in got:
        assert np.all(g[total:] == 7.0)                               # rows behind the last sequence


def test_read_bad_rows_and_first_none():
    s = oc.Shape(1, 128, 4, 32, True)
    c = Both(s, 2, 2, 4, bad=((1, 0, 77),))
    rng = np.random.default_rng(1)
    x = bf16(rng.standard_normal((80, 1, 128)))
    x[2, 0, 1] = np.nan
    c.set_lens([40, 40])
    c.append(x, x, [40, 40])
    out = c.torch.full((80, 1, 128), 3.0, device="cuda")
    out2 = out.clone()
    c.gpu.read(None, c.i32([0, 40, 80]), 40, out, out2)
    g = out.cpu().numpy()
    assert np.all(np.isnan(g[2])) and np.all(np.isfinite(np.delete(g[:40], 2, 0)))
    assert np.all(g[40:72] == 0) and np.all(np.isfinite(g[72:]))      # a page outside the pool reads as zeros


# ------------------------------------------------------------------ attention
def reference(c, b, n, q, scale, cap=0.0, slopes=None, window=0, prefix=0, first=None, tree=None, merge=None):
    """Reference rows of one sequence and their error bounds: o, lse, err_o (norms), err_lse."""
    s, T = c.s, c.ref.lens[b]
    k, ok = c.ref.rows(b, 0, T, False)
    v, _ = c.ref.rows(b, 0, T, True)
    ks, _ = c.ref.rows(b, 0, T, False, rotated=True)
    vs, _ = c.ref.rows(b, 0, T, True, rotated=True)
    sc, _ = c.ref.scales(b, T)
    vis = oc.visible(n, T, ok, window, prefix, first, tree)
    pos, tok = oc.positions(n, T, tree)
    o, lse, p = oc.attend(q, k, v, vis, pos, tok, scale, cap, slopes)
    G = q.shape[1] // s.H
    err_o, err_l = np.zeros(lse.shape), np.zeros(lse.shape)
    for j in range(q.shape[1]):
        h = j // G
        qr = oc.wht.rotate(q[:, j], oc.signs(s, False)) if s.rotate else q[:, j]
        aq = np.abs(qr)
        for i in range(n):
            idx = np.nonzero(vis[i])[0]
            if not len(idx):
                continue
            big = np.repeat(sc[idx, h], 64, axis=-1)
            ds = scale * (aq[i] * ((2.0 ** -16 if s.rotate else 0) * np.abs(ks[idx, h])
                                   + 2.0 ** -24 * (s.d + 4) * 264 * big)).sum(-1)
            if slopes is not None:
                ds = ds + 2.0 ** -22 * float(slopes[j]) * np.abs(pos[i] - tok[idx])
            if cap:
                ds = ds + cap * 2.0 ** -21
            delta = float(ds.max())
            tail = 2.0 ** -24 * (T / 16 + 70) + 2.0 ** -20
            A = p[i, j, idx] @ np.abs(vs[idx, h])
            err_o[i, j] = (2.0 ** -8 + 2 * delta + tail) * np.linalg.norm(A)
            err_l[i, j] = delta + tail + 2.0 ** -20 * (1 + abs(lse[i, j]))
    if merge is not None:
        o2, l2 = merge
        both = np.logaddexp(lse, l2)
        m = np.where(np.isneginf(both), 0.0, both)                    # nothing in either part: both weights 0
        w1, w2 = np.exp(lse - m), np.exp(l2 - m)
        err_l = np.where(np.isneginf(both), 0.0, err_l)
        err_o = w1 * err_o + 2 * (err_l + 2.0 ** -20) * (np.linalg.norm(o, axis=-1) + np.linalg.norm(o2, axis=-1))
        err_l = err_l + 2.0 ** -20 * (1 + np.abs(m))
        o, lse = o * w1[..., None] + o2 * w2[..., None], both
    return o, lse, err_o + 2.0 ** -8 * np.linalg.norm(o, axis=-1), err_l


def attend_and_check(c, n, G, scale=None, cap=0.0, slopes=False, window=0, prefix=None, first=None, tree=None,
                     merge=False, q=None, max_len=None, spare=3, run=None, lse_wanted=True, many=True):
    """many: once more with a bound on the rows that picks the kernel of many query columns, where one does."""
    s, t = c.s, c.torch
    hq, st = s.H * G, c.starts(n)
    total = int(st[-1])
    rng = np.random.default_rng(total + hq)
    scale = float(np.float32(s.d ** -0.5 if scale is None else scale))
    if q is None:
        q = bf16(rng.standard_normal((total + spare, hq, s.d)) * 1.5)
    out = t.full((total + spare, hq, s.d), 7.0, dtype=t.bfloat16, device="cuda")
    lse = t.full((total + spare, hq), 7.0, device="cuda") if lse_wanted else None
    kw = dict(scale=scale, cap=cap, window=window)
    sl = None
    if slopes:
        sl = (2.0 ** (-8.0 * (np.arange(hq) + 1) / hq)).astype(np.float32)
        kw["slopes"] = t.from_numpy(sl).cuda()
    if prefix is not None:
        kw["prefix"] = c.i32(prefix)
    if first is not None:
        kw["first"] = c.i32(list(first) + [0] * spare)
    if merge:
        mo = (rng.standard_normal((total + spare, hq, s.d)) * 0.5).astype(np.float32)
        ml = (rng.standard_normal((total + spare, hq)) + 4).astype(np.float32)
        ml[0, 0] = -np.inf
        kw["merge_out"], kw["merge_lse"] = t.from_numpy(mo).cuda(), t.from_numpy(ml).cuda()
    max_len = max(c.ref.lens) if max_len is None else max_len
    bounds = [int(max(n))]
    big = 64 if tree is not None else (1 << 17) // G
    if many and bounds[0] < big and big * G > 128:
        bounds.append(big)
    worst, refs = 0.0, {}
    for max_q in bounds:
        if max_q == big and tree is not None:
            max_len = max(max_len, 1 << 20)              # few columns: more scores make it the kernel of many
        args = [c.dev(q, "bf16"), c.i32(st), max_q, max_len]
        out.fill_(7.0)
        if lse_wanted:
            lse.fill_(7.0)
        if tree is not None:
            m = np.array([x for row in tree for x in row] + [0] * spare, dtype=np.uint64).view(np.int64)
            call = lambda: c.gpu.tree_attention(*args, t.from_numpy(m.copy()).cuda(), out, lse, **kw)  # noqa: E731
        else:
            call = lambda: c.gpu.attention(*args, out, lse, **kw)                                       # noqa: E731
        (run or (lambda f: f()))(call)
        t.cuda.synchronize()
        go = out.float().cpu().numpy().astype(np.float64)
        gl = lse.cpu().numpy().astype(np.float64) if lse_wanted else None
        for b in range(c.batch):
            r = slice(st[b], st[b + 1])
            if n[b] == 0:
                continue
            if b not in refs:
                refs[b] = reference(c, b, n[b], q[r].astype(np.float64), scale, cap, sl, window,
                                    0 if prefix is None else prefix[b], None if first is None else list(first)[r],
                                    None if tree is None else tree[b],
                                    (mo[r].astype(np.float64), ml[r].astype(np.float64)) if merge else None)
            o, l, eo, el = refs[b]
            none, bad = np.isneginf(l), np.isnan(o).any(-1)          # bad: a NaN row is visible
            assert np.all(go[r][none] == 0) and np.all(np.isnan(go[r][bad]))
            err, eo = np.linalg.norm(np.where(bad[..., None], 0, go[r] - o), axis=-1), np.where(bad, 0, eo)
            none |= bad
            assert np.all(err <= eo + 1e-30), (max_q, b, np.max(err / (eo + 1e-30)))
            worst = max(worst, float(np.max(err / (eo + 1e-30))))
            if lse_wanted:
                assert np.all(np.isneginf(gl[r][none & ~bad]))
                assert np.all(np.abs(gl[r][~none] - l[~none]) <= el[~none])
        assert np.all(go[total:] == 7.0) and (gl is None or np.all(gl[total:] == 7.0))
    return worst


def filled(shape, lens, seed=0, max_pages=None, dtype="bf16", bad=(), **kw):
    s = oc.Shape(*shape, seed=3)
    mp = max_pages or max(1, max((x + s.P - 1) // s.P for x in lens))
    c = Both(s, len(lens), mp, len(lens) * mp + 1, seed=seed, bad=bad)
    c.grow(list(lens), np.random.default_rng(seed + 1), dtype, **kw)
    return c


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_decode(shape):
    """One token a sequence over 1, 2, 31, 32, 33 and several hundred tokens."""
    c = filled(shape, [1, 2, 31, 32, 33, 300])
    for G in (1, 4):
        attend_and_check(c, [1] * 6, G)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 20])
def test_head_groups(G):
    c = filled((2, 128, 4, 64, True), [70, 9])
    attend_and_check(c, [3, 1], G)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_prompt_rows(shape):
    """Several rows a sequence, some sequences none, and rows that are all of their cache."""
    c = filled(shape, [90, 40, 17, 130])
    attend_and_check(c, [37, 0, 17, 5], 2)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_terms(shape):
    c = filled(shape, [150, 33, 100])
    n = [21, 4, 9]
    attend_and_check(c, n, 2, cap=5.0)
    attend_and_check(c, n, 2, slopes=True)
    attend_and_check(c, n, 2, window=13)
    attend_and_check(c, n, 2, window=1, cap=2.0)
    attend_and_check(c, n, 2, prefix=[5, 0, 200], window=20)
    attend_and_check(c, n, 2, prefix=[150, 33, 0])
    docs = np.concatenate([np.arange(l - x, l) // 10 * 10 for x, l in zip(n, c.ref.lens)])
    attend_and_check(c, n, 2, first=docs, slopes=True, cap=30.0, window=7, prefix=[3, 31, 96])
    attend_and_check(c, n, 2, merge=True, lse_wanted=True)
    attend_and_check(c, n, 2, lse_wanted=False)


@pytest.mark.parametrize("shape", SHAPES[:4], ids=IDS[:4])
def test_rows_that_see_nothing(shape):
    c = filled(shape, [64, 20])
    n = [6, 3]
    first = [64, 64, 61, 64, 0, 1000, 20, 0, 2 ** 31 - 1]
    attend_and_check(c, n, 2, first=first)
    attend_and_check(c, n, 2, first=[2 ** 30] * 9, prefix=[4, 4], merge=True)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_split_rows_many(shape):
    """The same for more query rows (the kernel of many columns), and few rows in many ranges."""
    c = filled(shape, [1700, 20, 1100])
    attend_and_check(c, [40, 20, 3], 2)
    attend_and_check(c, [33, 1, 2], 2, window=900, prefix=[3, 0, 70], merge=True, cap=10.0)
    attend_and_check(c, [1, 1, 1], 1, max_len=10 ** 6)
    attend_and_check(c, [70, 20, 3], 2, max_len=10 ** 6)         # many columns in ranges
    attend_and_check(c, [65, 1, 2], 2, window=900, prefix=[3, 0, 70], merge=True, cap=10.0, max_len=10 ** 5)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_split_rows(shape):
    """Caches long enough to be cut into ranges, joined by the second launch."""
    c = filled(shape, [1500, 700, 20])
    attend_and_check(c, [1, 1, 1], 4)
    attend_and_check(c, [2, 1, 3], 1, window=300, prefix=[40, 3, 0], merge=True)
    attend_and_check(c, [1, 2, 1], 2, slopes=True, cap=20.0, max_len=100000)   # more ranges than tokens
    attend_and_check(c, [1, 2, 1], 2, max_len=0)                               # none
    attend_and_check(c, [1, 1, 1], 2, first=[2000, 690, 3])


@pytest.mark.parametrize("scale", [1e-3, 1.0])
def test_large_and_small_scores(scale):
    c = filled((2, 128, 8, 64, False), [260, 50])
    attend_and_check(c, [2, 1], 2, scale=scale)


def test_running_maximum_rises():
    """Scores that climb by more than the rescaling step from block to block, and fall again."""
    for rising in (True, False):
        s = oc.Shape(1, 64, 8, 32, False)
        c = Both(s, 1, 12, 12)
        T = 380
        k = np.zeros((T, 1, 64), dtype=np.float32)
        ramp = np.linspace(-40, 40, T)
        k[:, 0, 0] = ramp if rising else ramp[::-1]
        v = bf16(np.random.default_rng(0).standard_normal((T, 1, 64)))
        c.set_lens([T])
        c.append(bf16(k), v, [T])
        q = np.zeros((1 + 3, 1, 64), dtype=np.float32)
        q[:, 0, 0] = 8.0
        attend_and_check(c, [1], 1, scale=0.5, q=q)


def test_garbage_in_masked_places():
    """NaN rows that no query sees change nothing; a visible one makes the row NaN."""
    s = oc.Shape(2, 128, 4, 32, True)
    c = Both(s, 1, 4, 4)
    x = bf16(np.random.default_rng(2).standard_normal((100, 2, 128)))
    x[10], x[50] = np.nan, np.inf
    c.set_lens([100])
    c.append(x, x, [100])
    attend_and_check(c, [4], 2, first=[51, 60, 96, 99])
    attend_and_check(c, [4], 2, window=49)
    out = c.torch.empty(1, 2, 128, dtype=c.torch.bfloat16, device="cuda")
    c.gpu.attention(c.dev(np.ones((1, 2, 128)), "bf16"), c.i32([0, 1]), 1, 100, out)
    assert bool(c.torch.isnan(out).all())


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("n", [3, 45])
def test_scales_far_apart(shape, n):
    """Huge and tiny rows: masked ones (another document, 1e20 times larger or smaller) change nothing
    for the rows that do not see them, and visible values of any size are summed in full."""
    s = oc.Shape(*shape, seed=3)
    for far in (1e20, 1e-20):
        c = Both(s, 1, (200 + s.P - 1) // s.P, 8, seed=1)
        rng = np.random.default_rng(7)
        k, v = (rng.standard_normal((200, s.H, s.d)) for _ in range(2))
        k[:75] *= far
        v[:75] *= far
        c.set_lens([200])
        c.append(bf16(k), bf16(v), [200])
        attend_and_check(c, [n], 2, first=[75] * n)
        attend_and_check(c, [n], 2, window=100)
        v = v * 2.0 ** rng.integers(-30, 30, (200, 1, 1))
        c.append(bf16(rng.standard_normal(k.shape)), bf16(v), [200])
        attend_and_check(c, [n], 2)
        attend_and_check(c, [n], 2, cap=4.0, slopes=True, first=[75] * n)


@pytest.mark.parametrize("n", [3, 45])
def test_zero_and_large_queries(n):
    for shape in (SHAPES[0], SHAPES[3], SHAPES[5]):
        c = filled(shape, [150, 80])
        rng = np.random.default_rng(n)
        q = bf16(rng.standard_normal((2 * n + 3, shape[0] * 2, shape[1])))
        q[::3] = 0
        attend_and_check(c, [n, n], 2, q=q)
        q[1::3] = bf16(q[1::3] * 1e-30)
        attend_and_check(c, [n, n], 2, q=q, cap=3.0, window=60)
        attend_and_check(c, [n, n], 2, q=bf16(q * 1e15), scale=1e-16)


def test_rows_and_keys_of_zeros():
    s = oc.Shape(2, 128, 4, 64, True)
    c = Both(s, 1, 4, 4)
    rng = np.random.default_rng(0)
    k, v = (bf16(rng.standard_normal((190, 2, 128))) for _ in range(2))
    k[:64], v[64:128] = 0, 0
    c.set_lens([190])
    c.append(k, v, [190])
    for n in (2, 40):
        attend_and_check(c, [n], 2)


def test_bad_pages_are_left_out():
    c = filled((2, 64, 8, 32, True), [120, 70], max_pages=4, bad=((0, 1, 1000), (0, 2, -1), (1, 0, -7)))
    attend_and_check(c, [3, 2], 2)
    attend_and_check(c, [30, 40], 2)
    c.set_lens([500, 70])                                       # longer than the table row
    out = c.torch.empty(2, 2, 64, dtype=c.torch.bfloat16, device="cuda")
    c.gpu.attention(c.dev(np.ones((2, 2, 64)), "bf16"), c.i32([0, 1, 2]), 1, 500, out)
    assert bool(c.torch.isfinite(out).all())


def test_strided_queries_and_outputs():
    """Queries inside a wider projection, outputs head-major."""
    c = filled((2, 128, 4, 64, True), [50])
    t = c.torch
    q = bf16(np.random.default_rng(1).standard_normal((5, 4, 128)))
    wide = t.zeros(5, 8, 128, dtype=t.bfloat16, device="cuda")
    wide[:, 2:6] = c.dev(q, "bf16")
    out = t.zeros(4, 5, 128, dtype=t.bfloat16, device="cuda").transpose(0, 1)
    ref = t.zeros(5, 4, 128, dtype=t.bfloat16, device="cuda")
    c.gpu.attention(wide[:, 2:6], c.i32([0, 5]), 5, 50, out)
    c.gpu.attention(c.dev(q, "bf16"), c.i32([0, 5]), 5, 50, ref)
    assert t.equal(out, ref)


# ------------------------------------------------------------------ trees
def random_tree(n, rng):
    parents = [int(rng.integers(-1, i)) for i in range(n)]
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | (1 << i))
    return m


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_tree(shape):
    lens, n = [90, 7, 64, 400], [13, 7, 64, 33]
    c = filled(shape, lens)
    rng = np.random.default_rng(9)
    tree = [random_tree(x, rng) for x in n]
    attend_and_check(c, n, 2, tree=tree)
    attend_and_check(c, n, 1, tree=tree, cap=10.0, slopes=True, window=9, prefix=[2, 0, 0, 30])
    attend_and_check(c, n, 1, tree=tree, merge=True)
    attend_and_check(c, n, 3, tree=tree, slopes=True, window=50, merge=True)


def test_tree_masks_of_nothing():
    c = filled((1, 64, 4, 32, True), [5, 40])
    attend_and_check(c, [5, 4], 2, tree=[[0, 2, 0, 8, 31], [1, 0, 4, 12]])


def test_chain_equals_decode():
    """A tree that is a chain gives what decoding its tokens one by one gives (the same sums up to
    their grouping: both within the bound of the same reference)."""
    s = oc.Shape(2, 128, 4, 32, True, seed=1)
    c = Both(s, 1, 4, 4)
    rng = np.random.default_rng(4)
    c.grow([50], rng)
    c.grow([6], rng)
    q = bf16(rng.standard_normal((6 + 3, 4, 128)))
    attend_and_check(c, [6], 2, tree=[[2 ** (i + 1) - 1 for i in range(6)]], q=q)
    for i in range(6):
        c.set_lens([51 + i])
        attend_and_check(c, [1], 2, q=np.concatenate([q[i:i + 1], q[6:]]))


# ------------------------------------------------------------------ keeping
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_keep_bytes(shape):
    s = oc.Shape(*shape, seed=8)
    c = Both(s, 4, 3, 13, seed=3)
    rng = np.random.default_rng(2)
    c.grow([29, 3, 0, 60], rng)
    base = list(c.ref.lens)
    c.grow([20, 1, 12, 30], rng)
    path = [[0, 2, 5, 19], [0], [11, 3, 3, 70, -1, 0], sorted(rng.permutation(30)[:17].tolist())]
    for b in range(4):
        c.ref.keep(base[b], path[b], b)
    c.gpu.keep(c.i32(base), c.i32(c.starts([len(p) for p in path])), c.i32([x for p in path for x in p]))
    c.check_pool()


def test_keep_left_out():
    s = oc.Shape(2, 64, 4, 32, False)
    c = Both(s, 3, 2, 7, bad=((0, 1, 50),))
    rng = np.random.default_rng(2)
    c.grow([30, 64, 10], rng)
    base, path = [28, 60, -3], [[1, 3, 5, 0], [3, 4, 5, 1, 0], [0, 1]]
    for b in range(2):
        c.ref.keep(base[b], path[b], b)
    c.gpu.keep(c.i32(base), c.i32(c.starts([4, 5, 2])), c.i32([x for p in path for x in p]))
    c.check_pool()


# ------------------------------------------------------------------ together
def test_speculative_run():
    """Prompt, drafted trees, kept paths, next steps: the pool stays the oracle's and every attention
    is within its bound; the last tail is read back as the rows that were kept."""
    s = oc.Shape(2, 128, 4, 64, True, seed=6)
    c = Both(s, 2, 4, 8, seed=5)
    rng = np.random.default_rng(7)
    c.grow([70, 33], rng)
    attend_and_check(c, [70, 33], 2)
    kept = []
    for step in range(3):
        base = list(c.ref.lens)
        n = [11, 6]
        c.grow(n, rng)
        attend_and_check(c, n, 2, tree=[random_tree(x, rng) for x in n])
        path = [[0, 3, 10], [0, 1, 4, 5]][::(1 if step % 2 else -1)]
        path = [[x for x in p if x < m] for p, m in zip(path, n)]
        for b in range(2):
            c.ref.keep(base[b], path[b], b)
        c.gpu.keep(c.i32(base), c.i32(c.starts([len(p) for p in path])), c.i32([x for p in path for x in p]))
        c.set_lens([x + len(p) for x, p in zip(base, path)])
        kept.append([len(p) for p in path])
        c.grow([1, 1], rng)
        attend_and_check(c, [1, 1], 2)
        c.check_pool()
    n = [4, 4]
    out = [c.torch.empty(8, 2, 128, device="cuda") for _ in range(2)]
    c.gpu.read(c.i32([x - 4 for x in c.ref.lens]), c.i32([0, 4, 8]), 4, out[0], out[1])
    for value, o in zip((False, True), out):
        want = np.concatenate([c.ref.rows(b, c.ref.lens[b] - 4, 4, value)[0] for b in range(2)])
        assert np.allclose(o.cpu().numpy(), want, rtol=0, atol=1e-5 * np.abs(want).max())


def test_joined_with_payload_attention():
    """The whole context: a compressed prefill (jolt_decode_attention over its payloads) and the
    tail's cache, joined; against fp64 attention over the payloads' rows and the cache's rows."""
    import synth
    from oracle import codec as ocodec, tucker
    from tests.gpu_util import payload_bytes, to_dev_bytes
    torch, jb = torch_cuda(), jolt_binding()
    L, H, T, d, G = 1, 2, 192, 128, 2
    cfg = synth.config("mistral7b_gqa_1k", L=L, H=H, T=T, d=d, rank_t=16, rank_f=12)
    dec, dev = [], []
    for it in synth.make_items(cfg, 2):
        sp = ocodec.stored_params(tucker.token_factor_exact(it.x, 16)[1], tucker.feature_factor(it.x)[1],
                                  tucker.core_full(it.x, tucker.token_factor_exact(it.x, 16)[1],
                                                   tucker.feature_factor(it.x)[1]), 16, 16, "bf16")
        enc = ocodec.encode(it.x, sp, 4, it.seed, it.item_id, "bf16")
        jit, al = jb.make_item(L, H, T, d, "bf16", it.item_id, it.seed), jb.jolt_alloc(16, 16, 4, 0, 0, 0.0)
        dev.append((jit, al, to_dev_bytes(payload_bytes(jb, jit, al, sp, "bf16", enc.words, enc.scale_bits), torch)))
        dec.append(oatt.decoded(enc, (L, H, T, d), it.seed, it.item_id, "bf16")[0])          # H, T, d
    c = filled((H, d, 4, 64, True), [45])
    q = bf16(np.random.default_rng(0).standard_normal((1, H * G, d)))
    scale = float(np.float32(d ** -0.5))
    o1 = torch.empty(1, H * G, d, device="cuda")
    l1 = torch.empty(1, H * G, device="cuda")
    qf = torch.from_numpy(q).cuda()
    grp = [jb.jolt_attn_group(dev[0][0], dev[1][0], dev[0][1], dev[1][1], dev[0][2].data_ptr(), dev[1][2].data_ptr(),
                              qf.data_ptr(), o1.data_ptr(), l1.data_ptr())]
    wsb = jb.jolt_attention_workspace_size(grp, H * G)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    jb.jolt_decode_attention(c.gpu.h, grp, H * G, scale, ws.data_ptr(), wsb, torch.cuda.current_stream().cuda_stream)
    out = torch.empty(1, H * G, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, H * G, device="cuda")
    c.gpu.attention(qf.bfloat16(), c.i32([0, 1]), 1, 45, out, lse, scale=scale, merge_out=o1, merge_lse=l1)
    k, v = (c.ref.rows(0, 0, 45, x)[0].transpose(1, 0, 2) for x in (False, True))
    for j in range(H * G):
        h = j // G
        o, l = oatt.softmax_attention(q[0, j:j + 1].astype(np.float64), np.concatenate([dec[0][h], k[h]]),
                                      np.concatenate([dec[1][h], v[h]]), scale)
        got = out[0, j].float().cpu().numpy()
        # the payload part is within 1e-4 (its own test's bound); the tail's weights and the output are bf16
        va = np.abs(np.concatenate([dec[1][h], v[h]])).max()
        assert np.linalg.norm(got - o[0]) <= 2.0 ** -7 * (np.linalg.norm(o[0]) + va * np.sqrt(d))
        assert abs(float(lse[0, j]) - l[0]) <= 1e-4 * (1 + abs(l[0]))


def test_captured_step_follows_lens():
    """Append and attention captured once and replayed with new rows, lengths and pages between replays."""
    s = oc.Shape(2, 128, 4, 32, True, seed=4)
    c = Both(s, 2, 20, 40)
    t = c.torch
    rng = np.random.default_rng(1)
    c.grow([500, 3], rng)
    k, v, q = (t.zeros(2, x, 128, dtype=t.bfloat16, device="cuda") for x in (2, 2, 4))
    out, lse = t.zeros(2, 4, 128, dtype=t.bfloat16, device="cuda"), t.zeros(2, 4, device="cuda")
    st = c.i32([0, 1, 2])
    ws = t.empty(c.gpu.workspace_bytes(2, 1, 600, 4), dtype=t.uint8, device="cuda")
    assert ws.numel() > 0

    def step():
        c.gpu.append(k, v, st, 1)
        c.gpu.attention(q, st, 1, 600, out, lse, workspace=ws)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    saved = c.pool.clone()
    with t.cuda.stream(side):
        step()
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    c.pool.copy_(saved)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    c.pool.copy_(saved)
    for i in range(5):
        kn, vn = (bf16(rng.standard_normal((2, 2, 128))) for _ in range(2))
        qn = bf16(rng.standard_normal((2, 4, 128)))
        c.set_lens([x + 1 for x in c.ref.lens])
        c.ref.append(kn, vn, [0, 1, 2])
        k.copy_(c.dev(kn, "bf16")), v.copy_(c.dev(vn, "bf16")), q.copy_(c.dev(qn, "bf16"))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        c.check_pool()
        eager, elog = t.zeros_like(out), t.zeros_like(lse)
        c.gpu.attention(q, st, 1, 600, eager, elog)
        assert t.equal(eager, out) and t.equal(elog, lse)
        for b in range(2):
            o, l, eo, el = reference(c, b, 1, qn[b:b + 1].astype(np.float64), float(np.float32(128 ** -0.5)))
            assert np.all(np.linalg.norm(out[b].float().cpu().numpy() - o[0], axis=-1) <= eo[0])
            assert np.all(np.abs(lse[b].cpu().numpy() - l[0]) <= el[0])


def test_streams_side_by_side():
    """Two streams over one cache, each with its own workspace, and repeated calls bit for bit."""
    c = filled((2, 128, 4, 64, True), [1800])
    t = c.torch
    q = c.dev(np.random.default_rng(0).standard_normal((1, 8, 128)), "bf16")
    outs = [t.zeros(1, 8, 128, dtype=t.bfloat16, device="cuda") for _ in range(8)]
    st = c.i32([0, 1])
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for i, o in enumerate(outs):
        with t.cuda.stream(streams[i % 2]):
            c.gpu.attention(q, st, 1, 1800, o)
    t.cuda.synchronize()
    assert len(c.gpu.workspaces) == 2
    for o in outs[1:]:
        assert t.equal(o, outs[0])


def test_captured_prompt_tree_keep_and_read():
    """A chunk of many query rows, a tree, its accepted path and the read captured in one graph, without a
    workspace of the caller's, and replayed with other contents and lengths between replays."""
    c = filled((2, 128, 4, 64, True), [1300, 900], max_pages=24)
    t, s = c.torch, c.s
    rng = np.random.default_rng(2)
    n, G = 40, 2
    k, v = (t.zeros(2 * n, s.H, s.d, dtype=t.bfloat16, device="cuda") for _ in range(2))
    q = t.zeros(2 * n, s.H * G, s.d, dtype=t.bfloat16, device="cuda")
    out, out2 = t.zeros_like(q), t.zeros_like(q)
    lse = t.zeros(2 * n, s.H * G, device="cuda")
    masks = t.tensor([(2 << i) - 1 for i in range(n)] * 2, dtype=t.int64, device="cuda")
    st, base, first = c.i32([0, n, 2 * n]), c.i32([0, 0]), c.i32([0, 0])
    kst, path = c.i32([0, 3, 5]), c.i32([0, 2, 3, 1, 30])
    rst = c.i32([0, 70, 100])
    rk, rv = (t.zeros(100, s.H, s.d, dtype=t.bfloat16, device="cuda") for _ in range(2))

    def step(o, l, o2, a, b):
        c.gpu.append(k, v, st, n)
        c.gpu.attention(q, st, n, 1400, o, l, window=700)
        c.gpu.attention(q, st, 1 << 16, 1400, o, l, window=700)
        c.gpu.attention(q, st, 100, 1 << 17, o, l, window=700)
        c.gpu.tree_attention(q, st, n, 1400, masks, o2)
        c.gpu.keep(base, kst, path)
        c.gpu.read(first, rst, 70, a, b)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step(out, lse, out2, rk, rv)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step(out, lse, out2, rk, rv)
    assert len(c.gpu.captured) > 0
    for i in range(4):
        lens = [1300 + 11 * i, 900 + 64 * i]
        c.lens.copy_(c.i32(lens))
        base.copy_(c.i32([x - n for x in lens]))
        first.copy_(c.i32([x - n - 20 for x in lens]))
        for x in (k, v, q):
            x.copy_(c.dev(rng.standard_normal(tuple(x.shape)), "bf16"))
        saved = c.pool.clone()
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        after = c.pool.clone()
        c.pool.copy_(saved)
        eager = [t.zeros_like(x) for x in (out, lse, out2, rk, rv)]
        step(*eager)
        t.cuda.synchronize()
        assert t.equal(after, c.pool)
        for x, y in zip(eager, (out, lse, out2, rk, rv)):      # bits: tokens never written may be NaN
            assert t.equal(x.view(t.int8), y.view(t.int8))


def test_two_graphs_replayed_side_by_side():
    c = filled((2, 128, 4, 64, True), [3000])
    t = c.torch
    st, q, outs, graphs = c.i32([0, 1]), [], [], []
    for i in range(2):
        q.append(c.dev(np.random.default_rng(i).standard_normal((1, 8, 128)), "bf16"))
        outs.append(t.zeros_like(q[i]))
    want = [t.zeros_like(x) for x in outs]
    for i in range(2):
        c.gpu.attention(q[i], st, 1, 3000, want[i])
    t.cuda.synchronize()
    for i in range(2):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            for _ in range(20):
                c.gpu.attention(q[i], st, 1, 3000, outs[i])
        graphs.append(g)
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(5):
        for i in range(2):
            outs[i].zero_()
        t.cuda.synchronize()
        for i in range(2):
            with t.cuda.stream(streams[i]):
                graphs[i].replay()
        t.cuda.synchronize()
        assert t.equal(outs[0], want[0]) and t.equal(outs[1], want[1])


@pytest.mark.parametrize("n", [1, 45])
def test_queries_that_are_not_numbers(n):
    """A row with an infinity or a NaN is NaN; the others do not change."""
    for shape in (SHAPES[0], SHAPES[5]):
        c = filled(shape, [150, 80])
        t, hq = c.torch, shape[0] * 2
        st, q = c.i32([0, n, 2 * n]), c.dev(np.random.default_rng(n).standard_normal((2 * n, hq, shape[1])), "bf16")
        clean, out = t.zeros_like(q), t.zeros_like(q)
        bound = 1 if n == 1 else 1 << 16
        c.gpu.attention(q, st, bound, 150, clean)
        q[0, 1, 5] = float("nan")
        q[n, 0, 60] = float("inf")
        c.gpu.attention(q, st, bound, 150, out)
        assert bool(out[0, 1].isnan().all()) and bool(out[n, 0].isnan().all())
        same = t.ones(2 * n, hq, dtype=t.bool, device="cuda")
        same[0, 1] = same[n, 0] = False
        # (a neighbour may raise its running maximum at another block: one rounding of weights and output)
        assert float((out - clean)[same].float().norm(dim=-1).max()) <= 2.0 ** -6 * float(clean.float().norm(dim=-1).max())


@pytest.mark.parametrize("G,bound", [(1, 1), (40, 1), (40, 1000), (40, 40000)])
def test_nan_rows_that_stand_alone(G, bound):
    """A visible NaN row is not lost where it is all that a row, a wave or a token range sees, nor where every
    other score is far above its part's."""
    for shape in (SHAPES[0], SHAPES[5]):
        s = oc.Shape(*shape, seed=3)
        for T, at in ((1, 0), (40, 39), (9000, 4500), (9000, 8999)):
            c = Both(s, 1, (T + s.P - 1) // s.P, (T + s.P - 1) // s.P)
            k, v = (bf16(np.random.default_rng(x).standard_normal((T, s.H, s.d))) for x in (1, 2))
            v[at, 0, 3] = np.nan
            q = bf16(np.random.default_rng(3).standard_normal((1, s.H * G, s.d)))
            k[at + 1:] += 100 * q[0, 0]
            c.set_lens([T])
            c.append(bf16(k), v, [T])
            t = c.torch
            out = t.zeros(1, s.H * G, s.d, dtype=t.bfloat16, device="cuda")
            c.gpu.attention(c.dev(q, "bf16"), c.i32([0, 1]), bound, T, out)
            nan = out.isnan()
            assert bool(nan[:, :G].all()) and not bool(nan[:, G:].any())


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[7]], ids=[IDS[0], IDS[7]])
def test_pages_past_4_gib(shape):
    """The same tokens in pages at the two ends of a pool of more than 2^32 bytes."""
    s = oc.Shape(*shape, seed=3)
    jb, t = jolt_binding(), torch_cuda()
    page = s.H * s.head_bytes
    pages = (1 << 32) // page + 40
    pool = t.zeros(pages * page, dtype=t.uint8, device="cuda")
    n, T, lens = 40, 500, None
    mp = (T + s.P - 1) // s.P
    rng = np.random.default_rng(1)
    k, v, q = (t.from_numpy(rng.standard_normal((x, h, s.d)).astype(np.float32)).cuda().bfloat16()
               for x, h in ((T, s.H), (T, s.H), (n, 2 * s.H)))
    starts, rows = (t.tensor([0, x], dtype=t.int32, device="cuda") for x in (T, n))
    lens = t.tensor([T], dtype=t.int32, device="cuda")
    got = []
    for low in (0, pages - mp):
        table = t.arange(low, low + mp, dtype=t.int32, device="cuda").view(1, mp)
        g = jb.JoltCache(s.H, s.d, s.bits, pool, table, lens, page_tokens=s.P, rotate=s.rotate, seed=3)
        g.append(k, v, starts, T)
        g.keep(t.tensor([T - 20], dtype=t.int32, device="cuda"), t.tensor([0, 2], dtype=t.int32, device="cuda"),
               t.tensor([4, 3], dtype=t.int32, device="cuda"))
        outs = [t.zeros_like(q), t.zeros_like(q[:1]), t.zeros_like(k), t.zeros_like(v)]
        g.attention(q, rows, 1 << 16, T, outs[0])
        g.attention(q[:1], t.tensor([0, 1], dtype=t.int32, device="cuda"), 1, T, outs[1])
        g.read(None, starts, T, outs[2], outs[3])
        t.cuda.synchronize()
        got.append(outs)
    assert bool(got[0][2].any()) and t.equal(pool[:mp * page], pool[(pages - mp) * page:])
    for x, y in zip(*got):
        assert t.equal(x, y)


def test_more_refusals():
    c = filled((2, 128, 4, 64, True), [20])
    t, jb = c.torch, c.jb
    st, q = c.i32([0, 1]), t.zeros(1, 4, 128, dtype=t.bfloat16, device="cuda")
    # 2 log2 e = 2.885 times scale, scale / cap and cap has to stay below 3.403e38
    for kw in (dict(scale=3e38), dict(scale=1.0, cap=8e-39), dict(scale=1.0, cap=3e38)):
        with pytest.raises(jb.JoltError) as e:
            c.gpu.attention(q, st, 1, 20, t.zeros_like(q), **kw)
        assert e.value.status == jb.JOLT_E_INVALID
    with pytest.raises(ValueError):
        c.gpu.attention(q, st, 1, 20, t.zeros_like(q), workspace=t.zeros(64, device="cuda"))


def test_empty_calls():
    s = oc.Shape(1, 64, 4, 32, True)
    c = Both(s, 1, 1, 1)
    t = c.torch
    e = t.empty(0, 1, 64, dtype=t.bfloat16, device="cuda")
    st = c.i32([0, 0])
    c.gpu.append(e, e, st, 0)
    c.gpu.read(None, st, 0, e, e)
    c.gpu.keep(c.i32([0]), st, c.i32([]))
    c.gpu.attention(e, st, 0, 0, e)
    # a row over a cache of no tokens
    c.set_lens([0])
    out, lse = t.ones(1, 2, 64, dtype=t.bfloat16, device="cuda"), t.ones(1, 2, device="cuda")
    c.gpu.attention(t.ones(1, 2, 64, dtype=t.bfloat16, device="cuda"), c.i32([0, 1]), 1, 0, out, lse)
    assert bool((out == 0).all()) and bool(t.isneginf(lse).all())


def test_refusals():
    c = filled((2, 128, 4, 64, True), [20])
    t, jb = c.torch, c.jb
    st = c.i32([0, 1])
    q = t.zeros(1, 4, 128, dtype=t.bfloat16, device="cuda")
    k = t.zeros(1, 2, 128, dtype=t.bfloat16, device="cuda")
    ok = dict(out=t.zeros_like(q))

    def status(f):
        with pytest.raises(jb.JoltError) as e:
            f()
        return e.value.status
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(cap=-1.0), dict(cap=float("inf")), dict(window=-1)):
        assert status(lambda: c.gpu.attention(q, st, 1, 20, **ok, **kw)) == jb.JOLT_E_INVALID
    assert status(lambda: c.gpu.attention(q, st, 1, 20, **ok, merge_lse=t.zeros(1, 4, device="cuda"))) == \
        jb.JOLT_E_INVALID
    assert status(lambda: c.gpu.attention(q[:, :3], st, 1, 20, t.zeros_like(q[:, :3]))) == jb.JOLT_E_INVALID
    assert status(lambda: c.gpu.attention(q, st, -1, 20, **ok)) == jb.JOLT_E_INVALID
    assert status(lambda: c.gpu.append(k, k, st, -1)) == jb.JOLT_E_INVALID
    assert status(lambda: c.gpu.tree_attention(q, st, 65, 20, t.zeros(1, dtype=t.int64, device="cuda"), **ok)) == \
        jb.JOLT_E_UNSUPPORTED
    small = t.zeros(16, dtype=t.uint8, device="cuda")
    assert status(lambda: c.gpu.attention(q, st, 1, 60000, **ok, workspace=small)) == jb.JOLT_E_WORKSPACE
    odd = t.zeros(1 * 4 * 128 + 4, dtype=t.bfloat16, device="cuda")[4:].view(1, 4, 128)
    assert status(lambda: c.gpu.attention(odd, st, 1, 20, **ok)) == jb.JOLT_E_INVALID
    assert status(lambda: c.gpu.read(None, st, 1, k.expand(1, 2, 128), k[:, :1].expand(1, 2, 128))) == jb.JOLT_E_INVALID
    with pytest.raises(ValueError):
        c.gpu.attention(q.float(), st, 1, 20, **ok)
    with pytest.raises(ValueError):
        c.gpu.attention(q, c.i32([0, 1, 2]), 1, 20, **ok)
    with pytest.raises(ValueError):
        c.gpu.append(k, k.float(), st, 1)
    with pytest.raises(ValueError):
        c.gpu.attention(q.cpu(), st, 1, 20, **ok)
    with pytest.raises(ValueError):
        jb.JoltCache(2, 128, 4, c.pool, c.table, c.lens[:0])
    with pytest.raises(jb.JoltError):
        jb.JoltCache(2, 128, 3, c.pool, c.table, c.lens)
