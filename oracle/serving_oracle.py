"""FP64 CPU oracle of the rotary and paged-cache operators.

TEST INFRASTRUCTURE ONLY, like flamia_oracle (whose E4M3 / E8M0 formats it
uses): rotary positions, the cache write (one exponent per 32-token block and
head, held codes rounded again where it grows; or one per token and head), the
read-back, softmax attention over cached values with a window and first
tokens, and the books of a pool of pages.  Sequences are walked one at a time over plain arrays: the cache is a
dict from (sequence, position) to rows, with no pages.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import flamia_oracle as O


def rope(x, pos, freqs, interleaved=False, mscale=1.0, inverse=False):
    """Rows x [T, H, d] at positions pos [T]: pair i turned by pos * freqs[i]."""
    x = np.asarray(x, dtype=np.float64)
    r = 2 * len(freqs)
    angle = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(freqs, dtype=np.float64)
    c, s = np.cos(angle) * mscale, np.sin(angle) * mscale
    if inverse:
        s = -s
    a = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    b = a + 1 if interleaved else a + r // 2
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def rope_axes(x, pos, axes, freqs, interleaved=False, mscale=1.0, inverse=False):
    """Rows x [T, H, d]: pair i turned by pos[axes[i]] * freqs[i], pos [axes, T].  Pairs of
    one axis are turned together, by rope with the other pairs' frequencies 0 (and their
    scale taken back)."""
    x = np.asarray(x, dtype=np.float64)
    axes, freqs = np.asarray(axes), np.asarray(freqs, dtype=np.float64)
    r = 2 * len(freqs)
    y = x.copy()
    for a in range(axes.max() + 1):
        z = rope(x, pos[a], np.where(axes == a, freqs, 0.0), interleaved, mscale, inverse)
        for i in np.nonzero(axes == a)[0]:
            for e in ((2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)):
                y[..., e] = z[..., e]
    return y


class Pages:
    """A pool's books and the arrays of its pages (numpy, first index the page), with
    the calls that change them, written as one step after another."""

    def __init__(self, page_size, table, refs, arrays):
        self.page, self.table, self.refs = page_size, np.array(table), np.array(refs)
        self.arrays = arrays

    def _use(self, p, by):
        if p >= 0:
            self.refs[p] += by

    def copy(self, src, dst):
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                for x in self.arrays:
                    x[b] = x[a]

    def fork(self, parents, children, lens):
        last = {c: (p, i) for i, (p, c) in enumerate(zip(parents, children)) if c >= 0}
        rows = {}
        for c, (p, _) in last.items():
            n = lens[p] if p >= 0 else 0
            row = np.full(self.table.shape[1], -1)
            need = -(-n // self.page)
            if need:
                row[:need] = self.table[p, :need]
            rows[c] = row, n
        for c, (row, n) in rows.items():
            for was, now in zip(self.table[c], row):
                self._use(was, -1)
                self._use(now, 1)
            self.table[c], lens[c] = row, n

    def reserve(self, n, starts):
        """False: not enough free pages (nothing changes)."""
        slots = [(b, j) for b, (c, s) in enumerate(zip(n, starts)) if c > 0
                 for j in range(s // self.page, (s + c - 1) // self.page + 1)]
        table, refs, copies = self.table.copy(), self.refs.copy(), []
        free = [p for p in range(len(refs)) if refs[p] == 0]
        # of a page whose users are all here the last one keeps it
        for b, j in slots:
            p = table[b, j]
            users = [s for s in slots if self.table[s] == p]
            keeps = p >= 0 and (self.refs[p] <= 1 or
                                (len(users) == self.refs[p] and users[-1] == (b, j)))
            if keeps:
                continue
            if not free:
                return False
            q = free.pop(0)
            if p >= 0:
                refs[p] -= 1
                copies.append((p, q, max(starts[b] - j * self.page, 0)))
            table[b, j], refs[q] = q, 1
        self.table, self.refs = table, refs
        for a, b, rows in copies:
            for x in self.arrays:
                x[b, :, :rows] = x[a, :, :rows]
        return True

    def compact(self):
        live = int((self.refs > 0).sum())
        for p in range(live, len(self.refs)):
            if self.refs[p] > 0:
                q = int(np.nonzero(self.refs == 0)[0][0])
                self.copy([p], [q])
                self.refs[q], self.refs[p] = self.refs[p], 0
                self.table[self.table == p] = q
        return live


class Cache:
    """K or V of several sequences: codes and scale bytes by position."""

    def __init__(self, nseq, H_kv, d, token_scales=False):
        self.codes = [np.zeros((0, H_kv, d), dtype=np.uint8) for _ in range(nseq)]
        self.scales = [np.zeros((0, H_kv), dtype=np.uint8) for _ in range(nseq)]
        self.token = token_scales

    def write(self, b, x, start):
        """Rows x [n, H_kv, d] of sequence b at positions start .. start + n."""
        x = np.asarray(x, dtype=np.float64)
        n, H, d = x.shape
        bad = ~np.isfinite(x)
        x = np.where(bad, 0.0, x)
        have = max(len(self.codes[b]), start + n)
        for name, fill in (("codes", (H, d)), ("scales", (H,))):
            old = getattr(self, name)[b]
            new = np.zeros((have,) + fill, dtype=np.uint8)
            new[:len(old)] = old
            getattr(self, name)[b] = new
        codes, scales = self.codes[b], self.scales[b]
        size = 1 if self.token else 32
        p = start
        while p < start + n:
            p0 = p // size * size
            end = min(p0 + size, start + n)
            new = x[p - start:end - start]
            e = O.roundup_exponent(np.abs(new).max(axis=(0, 2)))  # [H]
            if p > p0:  # (rows that were written again may have exponents of their own)
                was = scales[p0:p].astype(int) - 127  # [held, H]
                e = np.maximum(e, was.max(axis=0))
                for r, h in np.argwhere(was < e):
                    held = codes[p0 + r, h]
                    nan = (held & 0x7F) == 0x7F
                    value = np.where(nan, 0.0, O.e4m3_decode(np.where(nan, 0, held)))
                    again = O.e4m3_encode(value * 2.0 ** float(was[r, h] - e[h]))
                    codes[p0 + r, h] = np.where(nan, 0x7F, again)
                    scales[p0 + r, h] = e[h] + 127
            c = O.e4m3_encode(new * np.ldexp(1.0, -e)[None, :, None])
            codes[p:end] = np.where(bad[p - start:end - start], 0x7F, c)
            scales[p:end] = (e + 127).astype(np.uint8)
            p = end

    def values(self, b):
        """Cached values of sequence b, float64 [L, H_kv, d]."""
        c = self.codes[b]
        nan = (c & 0x7F) == 0x7F
        v = O.e4m3_decode(np.where(nan, 0, c)) * O.e8m0_decode(self.scales[b])[:, :, None]
        return np.where(nan, np.nan, v)


def seen_keys(p, L, window=0, sinks=0):
    """Mask over keys 0 .. L-1 of a query at position p."""
    j = np.arange(L)
    m = j <= p
    if window > 0:
        m &= (j > p - window) | (j < sinks)
    return m


def attend(q, k, v, start, scale, window=0, sinks=0, v_exponents=None):
    """(o [n, H, d], lse [H, n]) of one sequence: queries q [n, H, d] at
    positions start .. over cached values k, v [L, H_kv, d].

    With v_exponents [L, H_kv] (those of v's scales) also what an error bound
    needs: mass [n, H, d] = sum p |v|, and top [n, H], the largest p 448 2^e of a
    seen key, exponents more than 60 below the largest seen counting as that."""
    q = np.asarray(q, dtype=np.float64)
    n, H, d = q.shape
    G = H // k.shape[1]
    o, lse = np.zeros((n, H, d)), np.full((H, n), -math.inf)
    mass, top = np.zeros((n, H, d)), np.zeros((n, H))
    for i in range(n):
        m = seen_keys(start + i, len(k), window, sinks)
        if not m.any():
            continue
        for h in range(H):
            x = k[m, h // G] @ q[i, h] * scale
            high = x.max()
            w = np.exp(x - high)
            o[i, h] = w @ v[m, h // G] / w.sum()
            lse[h, i] = high + math.log(w.sum())
            if v_exponents is not None:
                e = v_exponents[m, h // G].astype(np.float64)
                mass[i, h] = w @ np.abs(v[m, h // G]) / w.sum()
                top[i, h] = (w * np.exp2(np.maximum(e, e.max() - 60))).max() * 448 / w.sum()
    return (o, lse) if v_exponents is None else (o, lse, mass, top)
