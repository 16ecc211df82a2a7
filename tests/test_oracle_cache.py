"""Pins for the token cache's oracle (oracle/cache.py): the page layout covers
every byte once, codes survive a round trip, and attention's masks mean what
their definitions say."""
import numpy as np
import pytest

from oracle import cache as oc


@pytest.mark.parametrize("d,bits,P", [(64, 4, 32), (64, 8, 64), (128, 4, 64), (128, 8, 32)])
def test_layout_covers_every_byte_once(d, bits, P):
    s = oc.Shape(1, d, bits, P, False)
    pg = oc.Pages(s, np.zeros(s.head_bytes, dtype=np.uint8))
    used = np.zeros(s.head_bytes * 2, dtype=int)                    # nibbles
    for value in (False, True):
        for t in range(P):
            for f in range(d):
                o, sh = pg._at(t, f, value)
                for x in range(bits // 4):
                    used[2 * o + sh // 4 + x] += 1
            for g in range(d // 64):
                o = pg._scale_at(t, g, value)
                used[2 * o:2 * o + 4] += 1
    assert np.all(used == 1)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rotate", [False, True])
def test_round_trip_error_is_half_a_step(bits, rotate):
    """|x~ - y| <= scale / 2 in the stored domain, plus what bf16 scales and clamping give up."""
    s = oc.Shape(2, 128, bits, 32, rotate, seed=3)
    x = np.random.default_rng(bits).standard_normal((40, 2, 128)).astype(np.float32)
    pool = np.full((2, 2, s.head_bytes), 0xA5, dtype=np.uint8)
    c = oc.Cache(s, pool, [[1, 0]], [40])
    c.append(x, x, [0, 40])
    for value in (False, True):
        r, ok = c.rows(0, 0, 40, value)
        assert ok.all()
        u, sb = oc.quantize_rows(s, x, value)
        assert np.array_equal(oc.values(s, u, sb, value), r)
        step = oc.quant.bf16_bits_to_f32(sb).max()
        # clamped values are at most qmax * 2^-8 of a step off on top of the half
        lim = step * (0.5 + oc.quant.qmax_for(bits) * 2.0 ** -8) * (np.sqrt(128) if rotate else 1)
        assert np.abs(r - x).max() <= lim


def test_zero_and_bad_rows():
    s = oc.Shape(1, 64, 4, 32, True)
    x = np.zeros((4, 1, 64), dtype=np.float32)
    x[1, 0, 3] = np.nan
    x[2, 0, 5] = np.inf
    x[3] = 1e-45
    u, sb = oc.quantize_rows(s, x, False)
    r = oc.values(s, u, sb, False)
    assert np.all(r[0] == 0) and np.all(np.isnan(r[1])) and np.all(np.isnan(r[2])) and np.all(r[3] == 0)


def test_masks():
    ok = np.ones(10, dtype=bool)
    v = oc.visible(3, 10, ok)
    assert [list(np.nonzero(r)[0]) for r in v] == [list(range(8)), list(range(9)), list(range(10))]
    v = oc.visible(1, 10, ok, window=3, prefix=2)
    assert list(np.nonzero(v[0])[0]) == [0, 1, 7, 8, 9]
    v = oc.visible(2, 10, ok, first=[4, 9], prefix=10)
    assert [list(np.nonzero(r)[0]) for r in v] == [[4, 5, 6, 7, 8, 9], [9]]
    # a chain is causal; two branches do not see each other
    v = oc.visible(3, 10, ok, tree=[0b001, 0b011, 0b101])
    assert [list(np.nonzero(r)[0]) for r in v] == [list(range(8)), list(range(9)), list(range(8)) + [9]]
    pos, tok = oc.positions(3, 10, [0b001, 0b011, 0b101])
    assert list(pos) == [7, 8, 8] and list(tok[7:]) == [7, 8, 8]
    # within a window, a slot counts by its depth
    v = oc.visible(3, 10, ok, window=2, tree=[0b001, 0b011, 0b101])
    assert [list(np.nonzero(r)[0]) for r in v] == [[6, 7], [7, 8], [7, 9]]


def test_keep_moves_in_any_order():
    s = oc.Shape(1, 64, 8, 32, False)
    x = np.arange(40 * 64, dtype=np.float32).reshape(40, 1, 64)
    pool = np.zeros((2, 1, s.head_bytes), dtype=np.uint8)
    c = oc.Cache(s, pool, [[0, 1]], [40])
    c.append(x, -x, [0, 40])
    before, _ = c.rows(0, 0, 40, True)
    c.keep(30, [1, 0, 9, 9], 0)
    after, _ = c.rows(0, 0, 40, True)
    want = before.copy()
    want[30:34] = before[[31, 30, 39, 39]]
    assert np.array_equal(after, want)
