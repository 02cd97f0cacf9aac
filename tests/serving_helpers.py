"""Shared by the GPU tests of the rotary and cache operators: page tables, the
cache of a list of sequences on the GPU and in the oracle, tolerances."""
import math

import numpy as np
import torch

from oracle import serving_oracle as S

DEV = "cuda"


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def offsets(n):
    return i32(np.concatenate([[0], np.cumsum(n)]))


def bf16(rng, shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.bfloat16)


def page_table(rng, lens, page, spare=3, width=None):
    """(table, pages): every sequence's pages scattered over the pool, -1 where none is
    needed; `spare` pages belong to nobody."""
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    t = np.full((len(lens), max([1] + need) if width is None else width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, pages


class Pair:
    """A GPU cache and the oracle's, fed with the same rows."""

    def __init__(self, fl, rng, lens, page, H_kv, d, token=False, fill=0x7F, width=None):
        self.t, pages = page_table(rng, lens, page, width=width)
        self.table = torch.from_numpy(self.t).to(DEV)
        self.gpu = fl.KVCache(pages, page, H_kv, d, token_scales=token)
        # what lies in pages before they are written: NaN codes, large scales
        for x in (self.gpu.k_codes, self.gpu.v_codes):
            x.fill_(fill)
        for x in (self.gpu.k_scales, self.gpu.v_scales):
            x.fill_(0xFE)
        self.k = S.Cache(len(lens), H_kv, d, token)
        self.v = S.Cache(len(lens), H_kv, d, token)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def write(self, k, v, n, starts):
        self.gpu.write(k.to(DEV), v.to(DEV), offsets(n), i32(starts), self.table,
                       dev_status=self.status)
        at = 0
        for b, c in enumerate(n):
            if c:
                self.k.write(b, k[at:at + c].double().numpy(), starts[b])
                self.v.write(b, v[at:at + c].double().numpy(), starts[b])
            at += c

    def gathered(self, b, n):
        """Codes and scale bytes of sequence b's first n positions: k, ks, v, vs."""
        page = self.gpu.page_size
        p = np.arange(n)
        pg, off = self.t[b, p // page], p % page
        return [x.cpu().numpy()[pg, :, off] for x in (self.gpu.k_codes, self.gpu.k_scales,
                                                      self.gpu.v_codes, self.gpu.v_scales)]

    def check_equal(self, lens):
        for b, n in enumerate(lens):
            k, ks, v, vs = self.gathered(b, n)
            for name, got, want in (("k", k, self.k.codes[b]), ("k scales", ks, self.k.scales[b]),
                                    ("v", v, self.v.codes[b]), ("v scales", vs, self.v.scales[b])):
                assert np.array_equal(got, want[:n]), (name, b)


def weight_error(T, nseq, G):
    """Relative rounding of a softmax weight: three E4M3 terms of 4 bits hold it
    to 2^-14; items of 16 or 32 rows (more than 8 rows a sequence and K / V head on
    average) round it to FP16 first, half a step of which is 2^-11, and its terms
    hold those 11 bits (E4M3, E4M3 and the 3 bits of E5M2); items of 256 rows multiply
    it as FP16."""
    return 2.0 ** -11 if -(-T // nseq) * G > 8 else 2.0 ** -14


def attend_tolerance(q, k, scale, n_keys, o, weight, mass, top):
    """How far an output of the cached attention may be off, elementwise: its BF16
    rounding (half a step, 2^-8 of the value), the relative error of the softmax
    weights (twice: the sum that divides them has it too) times mass = sum p |v|,
    and 2^-24 of the largest weight times value scale (top) for each key below
    the weights' range.  A score is off by at most 2^-19.5 + 2^-17 of scale |q| |k|
    (the query's split into E4M3 terms; float32 sums of d exact products), taken
    as 2^-16; a weight by twice that, by `weight` (its own split into terms) and
    2^-20 for exp2 and the sums."""
    qn = np.sqrt((q ** 2).sum(-1)).max()
    kn = np.sqrt((k ** 2).sum(-1)).max()
    rel = 2 * 2.0 ** -16 * scale * qn * kn + weight + 2.0 ** -20
    return 2.0 ** -8 * np.abs(o) + 2 * rel * mass + 2 * n_keys * 2.0 ** -24 * top


def lse_tolerance(q, k, scale, lse):
    qn = np.sqrt((q ** 2).sum(-1)).max()
    kn = np.sqrt((k ** 2).sum(-1)).max()
    return 2.0 ** -16 * scale * qn * kn + 2.0 ** -20 * (1 + np.abs(lse))


def check_attend(o, lse, pair, q, n, starts, scale, window=0, sinks=0):
    """Rows of every sequence against the oracle."""
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    at = 0
    for b, c in enumerate(n):
        if c == 0:
            continue
        qb = q[at:at + c].double().cpu().numpy()
        k, v = pair.k.values(b)[:max(starts[b], 0) + c], pair.v.values(b)[:max(starts[b], 0) + c]
        e = pair.v.scales[b][:len(k)].astype(int) - 127
        ro, rl, mass, top = S.attend(qb, k, v, starts[b], scale, window, sinks, e)
        tol = attend_tolerance(qb, k, scale, len(k), ro,
                               weight_error(len(q), len(n), q.shape[1] // pair.gpu.H_kv), mass,
                               top[..., None])
        got, gl = o[at:at + c], lse[:, at:at + c]
        assert np.isfinite(got).all(), ("o", b)
        worst = np.max(np.abs(got - ro) / np.maximum(tol, 2.0 ** -133))  # (BF16's smallest step)
        assert worst <= 1, ("o", b, worst, np.abs(got - ro).max())
        none = rl == -math.inf
        assert np.array_equal(none, gl == -math.inf)
        assert (got.transpose(1, 0, 2)[none] == 0).all()
        if (~none).any():
            err = np.abs(gl[~none] - rl[~none]) / lse_tolerance(qb, k, scale, rl[~none])
            assert err.max() <= 1, ("lse", b, err.max())
        at += c
