"""ORACLE (test infrastructure only): the token cache, plainly, in fp64 numpy.

Rows are quantized with the codec's own steps (quant.quantize_groups, fp32 by
definition) after the rotation summed in fp64 and rounded to fp32 once; pages
are plain byte arrays filled member by member; attention is the textbook
softmax over the rows the pages stand for.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from . import quant, rng, wht

GROUP = quant.GROUP


@dataclass
class Shape:
    H: int
    d: int
    bits: int
    P: int
    rotate: bool
    seed: int = 0
    k_id: int = 0
    v_id: int = 1

    @property
    def code_bytes(self):
        return self.P * self.d * self.bits // 8

    @property
    def scale_bytes(self):
        return self.P * (self.d // GROUP) * 2

    @property
    def head_bytes(self):
        return 2 * self.code_bytes + 2 * self.scale_bytes


def signs(s: Shape, value: bool):
    return rng.rotation_signs(s.seed, s.v_id if value else s.k_id, s.d)


def quantize_rows(s: Shape, x: np.ndarray, value: bool):
    """x (..., d) fp32 -> codes (..., d) uint8 and scale bits (..., d / 64) uint16."""
    y = np.asarray(x, dtype=np.float32)
    if s.rotate:
        with np.errstate(invalid="ignore", over="ignore"):
            y = (wht.fwht(y.astype(np.float64) * signs(s, value)) * (1.0 / np.sqrt(s.d))).astype(np.float32)
    bad = ~np.all(np.isfinite(y), axis=-1)
    y = np.where(bad[..., None], np.float32(0), y)
    g = y.reshape(y.shape[:-1] + (s.d // GROUP, GROUP))
    tiny = quant.f32_to_bf16_bits(np.max(np.abs(g), axis=-1) / np.float32(quant.qmax_for(s.bits))) < 0x0080
    g = np.where(tiny[..., None], np.float32(0), g)
    q, sb = quant.quantize_groups(g, s.bits)
    sb = np.where(bad[..., None], np.uint16(0x7FC0), sb).astype(np.uint16)
    u = quant.codes_from_q(q, s.bits).astype(np.uint8).reshape(y.shape)
    return u, sb


def values(s: Shape, u, sb, value: bool, rotated: bool = False):
    """fp64 rows the codes stand for (rotated: as they are stored)."""
    q = u.astype(np.float64) - (1 << (s.bits - 1))
    with np.errstate(invalid="ignore"):
        x = (q.reshape(q.shape[:-1] + (s.d // GROUP, GROUP))
             * quant.bf16_bits_to_f32(sb).astype(np.float64)[..., None]).reshape(q.shape)
    if s.rotate and not rotated:
        x = wht.unrotate(x, signs(s, value))
    return x


class Pages:
    """The pool as bytes [pages][H][head_bytes], with one token's members put and got one by one."""

    def __init__(self, s: Shape, pool: np.ndarray):
        self.s, self.pool = s, pool.reshape(-1, s.H, s.head_bytes)

    def _at(self, t_in, f, value):
        """Byte offset and bit shift of a code."""
        s = self.s
        if value:
            unit, e = (t_in // 8) * s.d + f, t_in % 8
        else:
            k, g, e = f // 32, (f % 32) // 8, f % 8
            unit = t_in * (s.d // 8) + g * (s.d // 32) + k
        base = s.code_bytes if value else 0
        if s.bits == 8:
            return base + unit * 8 + e, 0
        nib = e // 2 + 4 * (e % 2)
        return base + unit * 4 + nib // 2, 4 * (nib % 2)

    def _offsets(self, t_in, value):
        ob = [self._at(t_in, f, value) for f in range(self.s.d)]
        return np.array([o for o, _ in ob]), np.array([b for _, b in ob])

    def _scale_at(self, t_in, g, value):
        s = self.s
        return 2 * s.code_bytes + (s.scale_bytes if value else 0) + 2 * (g * s.P + t_in)

    def put(self, page, t_in, u, sb, value):
        """u (H, d), sb (H, d / 64)."""
        s = self.s
        off, sh = self._offsets(t_in, value)
        p = self.pool[page]
        if s.bits == 8:
            p[:, off] = u
        else:
            for o, b, c in zip(off, sh, u.T):
                p[:, o] = (p[:, o] & (0xF0 >> b)) | (c << b)
        for g in range(s.d // GROUP):
            o = self._scale_at(t_in, g, value)
            p[:, o] = sb[:, g] & 255
            p[:, o + 1] = sb[:, g] >> 8

    def get(self, page, t_in, value):
        s = self.s
        off, sh = self._offsets(t_in, value)
        p = self.pool[page]
        u = p[:, off] if s.bits == 8 else (p[:, off] >> sh) & 15
        sb = np.stack([p[:, self._scale_at(t_in, g, value)].astype(np.uint16)
                       | (p[:, self._scale_at(t_in, g, value) + 1].astype(np.uint16) << 8)
                       for g in range(s.d // GROUP)], -1)
        return u.astype(np.uint8), sb


class Cache:
    """Pool, page table and lengths; page numbers outside the pool lose their tokens."""

    def __init__(self, s: Shape, pool, table, lens):
        self.s, self.pages, self.table, self.lens = s, Pages(s, pool), np.asarray(table), list(lens)

    def place(self, b, t):
        p = t // self.s.P
        if t < 0 or p >= self.table.shape[1]:
            return None
        page = int(self.table[b, p])
        return (page, t % self.s.P) if 0 <= page < self.pages.pool.shape[0] else None

    def append(self, k, v, starts):
        """k, v (total, H, d) fp32; lens already count the new rows."""
        coded = [quantize_rows(self.s, x, value) for x, value in ((k, False), (v, True))]
        for b in range(len(self.lens)):
            n = starts[b + 1] - starts[b]
            for i in range(n):
                at = self.place(b, self.lens[b] - n + i)
                if at is None:
                    continue
                for value, (u, sb) in zip((False, True), coded):
                    self.pages.put(at[0], at[1], u[starts[b] + i], sb[starts[b] + i], value)

    def rows(self, b, t0, n, value, rotated=False):
        """fp64 rows (n, H, d) of tokens t0 .. and which of them exist."""
        s = self.s
        u = np.full((n, s.H, s.d), 1 << (s.bits - 1), dtype=np.uint8)
        sb = np.zeros((n, s.H, s.d // GROUP), dtype=np.uint16)
        ok = np.zeros(n, dtype=bool)
        for i in range(n):
            at = self.place(b, t0 + i) if 0 <= t0 + i < self.lens[b] else None
            if at is not None:
                u[i], sb[i] = self.pages.get(at[0], at[1], value)
                ok[i] = True
        return values(s, u, sb, value, rotated), ok

    def scales(self, b, n):
        """fp64 K and V scales (n, H, d / 64), zeros where the token is missing."""
        out = []
        for value in (False, True):
            sb = np.zeros((n, self.s.H, self.s.d // GROUP), dtype=np.uint16)
            for t in range(n):
                at = self.place(b, t)
                if at is not None:
                    sb[t] = self.pages.get(at[0], at[1], value)[1]
            out.append(quant.bf16_bits_to_f32(sb).astype(np.float64))
        return out

    def keep(self, base, path, b):
        src = [self.place(b, base + p) if 0 <= p < 64 else None for p in path]
        rows = [None if at is None else [self.pages.get(at[0], at[1], value) for value in (False, True)] for at in src]
        for i, r in enumerate(rows[:64]):
            at = self.place(b, base + i)
            if r is None or at is None:
                continue
            for value, (u, sb) in zip((False, True), r):
                self.pages.put(at[0], at[1], u, sb, value)


def positions(n, length, tree=None):
    """Positions of the n query rows and of all tokens (tree: lists of bit masks)."""
    base = length - n
    tok = np.arange(length)
    if tree is None:
        return base + np.arange(n), tok
    depth = np.array([max(bin(int(m)).count("1") - 1, 0) for m in tree])
    tok = tok.copy()
    tok[base:] = base + depth
    return base + depth, tok


def visible(n, length, ok, window=0, prefix=0, first=None, tree=None):
    base = length - n
    pos, tok = positions(n, length, tree)
    out = np.zeros((n, length), dtype=bool)
    for i in range(n):
        for t in range(length):
            if not ok[t]:
                continue
            inside = window == 0 or pos[i] - tok[t] < window
            if tree is not None and t >= base:
                out[i, t] = bool((int(tree[i]) >> (t - base)) & 1) and inside
            else:
                out[i, t] = t >= (first[i] if first is not None else 0) and \
                    (t < prefix or (t <= pos[i] and (tree is not None or t <= base + i) and inside))
    return out


def attend(q, k, v, vis, pos, tok, scale, cap=0.0, slopes=None):
    """q (n, hq, d); k, v (T, H, d); vis (n, T).  Returns o (n, hq, d), lse (n, hq), p (n, hq, T)."""
    n, hq, d = q.shape
    H = k.shape[1]
    G = hq // H
    o, lse, pw = np.zeros((n, hq, d)), np.full((n, hq), -np.inf), np.zeros((n, hq, k.shape[0]))
    for j in range(hq):
        kk, vv = k[:, j // G], v[:, j // G]
        for i in range(n):
            idx = np.nonzero(vis[i])[0]
            if len(idx) == 0:
                continue
            s = scale * (kk[idx] @ q[i, j])
            if cap:
                s = cap * np.tanh(s / cap)
            if slopes is not None:
                s = s - float(slopes[j]) * np.abs(pos[i] - tok[idx])
            m = np.max(s)
            w = np.exp(s - m)
            pw[i, j, idx] = w / w.sum()
            o[i, j] = (w / w.sum()) @ vv[idx]
            lse[i, j] = m + np.log(w.sum())
    return o, lse, pw
