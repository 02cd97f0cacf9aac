"""Attention over the cache with a shared prefix against the oracle, which knows of
none: every sequence's own keys and values, row by row."""
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.serving_helpers import DEV, Pair, attend_tolerance, bf16, i32, lse_tolerance, offsets

pytestmark = pytest.mark.gpu


class Forked(Pair):
    """Sequences of `prefix` common tokens and own[b] of their own (0: none at all).  Each
    has written all of them into its own pages; those of the whole tiles of the prefix are
    then taken from every table row but that of the first sequence that shares it, so that
    a kernel which looks for them there reports it."""

    def __init__(self, fl, rng, prefix, own, page, H_kv, d, scale=1.0, token=False):
        lens = [prefix + n if n else 0 for n in own]
        super().__init__(fl, rng, lens, page, H_kv, d, token)
        self.lens, self.prefix = lens, prefix
        self.x = [bf16(rng, (prefix, H_kv, d), scale) for _ in range(2)]
        self.y = [bf16(rng, (sum(own), H_kv, d), scale) for _ in range(2)]
        k, v = (torch.cat([t for at, n in zip(np.cumsum([0] + list(own)), own) if n
                           for t in (x, y[at:at + n])]) for x, y in zip(self.x, self.y))
        self.write(k, v, lens, [0] * len(lens))

    def share(self, n, starts):
        first = True
        for b, c in enumerate(n):
            if c and starts[b] >= self.prefix - 1:
                if not first:
                    self.t[b, :self.prefix // 128 * 128 // self.gpu.page_size] = -1
                first = False
        self.table.copy_(torch.from_numpy(self.t))


def _check(o, lse, pair, q, n, starts, scale):
    """As check_attend, with the rounding of the form that takes the prefix: rows of 16
    and more multiply weights rounded to FP16 (2^-11)."""
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    T, G = sum(n), q.shape[1] // pair.gpu.H_kv
    weight = 2.0 ** -11 if T * G > 8 else 2.0 ** -14
    at = 0
    for b, c in enumerate(n):
        if c == 0:
            continue
        qb = q[at:at + c].double().cpu().numpy()
        end = max(starts[b], 0) + c
        k, v = pair.k.values(b)[:end], pair.v.values(b)[:end]
        e = pair.v.scales[b][:end].astype(int) - 127
        ro, rl, mass, top = S.attend(qb, k, v, starts[b], scale, v_exponents=e)
        tol = attend_tolerance(qb, k, scale, len(k), ro, weight, mass, top[..., None])
        got, gl = o[at:at + c], lse[:, at:at + c]
        none = rl == -math.inf
        assert np.isfinite(got).all(), b
        assert (np.abs(got - ro) <= np.maximum(tol, 2.0 ** -133)).all(), (b, (np.abs(got - ro) / tol).max())
        assert np.array_equal(none, gl == -math.inf)
        assert (got.transpose(1, 0, 2)[none] == 0).all()
        assert (np.abs(gl[~none] - rl[~none]) <= lse_tolerance(qb, k, scale, rl[~none])).all(), b
        at += c


def _run(fl, pair, rng, H, n, starts, prefix, T=None, scale=None, q=None):
    d = pair.gpu.d
    T = sum(n) if T is None else T
    scale = d ** -0.5 if scale is None else scale
    q = bf16(rng, (T, H, d)).to(DEV) if q is None else q
    o = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((H, T), 7.0, device=DEV)
    pair.gpu.attend(q, offsets(n), i32(starts), pair.table, scale, prefix=prefix, o=o, lse=lse,
                    dev_status=pair.status, always_share=True)
    return q, o, lse, scale


@pytest.mark.parametrize("H,H_kv,d,page,prefix,own,n", [
    # (rows of the prefix, of a sequence) = 2, 4, 8; 1
    (1, 1, 64, 32, 128, [1, 3], [1, 1]),
    (2, 1, 128, 64, 300, [5, 40], [1, 1]),
    (4, 4, 64, 64, 1000, [1, 130, 64, 7, 2, 33, 1, 129], [1] * 8),
    # 9 .. 16; 4 and 8 rows a sequence
    (8, 2, 128, 32, 517, [9, 1, 260], [1, 1, 1]),
    (8, 1, 64, 128, 640, [300, 2], [1, 1]),
    # 32 rows: 20, 17 and 32, sequences of 4, 1, 8 and 16
    (16, 4, 128, 256, 1291, [17, 400, 3, 90, 1], [1] * 5),
    (2, 2, 64, 64, 700, [1 + 30 * (i % 5) for i in range(17)], [1] * 17),
    (8, 1, 64, 128, 515, [1, 300, 44, 7], [1] * 4),
    (8, 2, 128, 32, 4000, [4, 200], [4, 4]),
    # 33 rows (two items of 32), and with 256 an item 69, 96, 97, 128, 200, 256, 260 and 520,
    # one to 32 a sequence
    (1, 1, 128, 32, 400, [1 + i for i in range(33)], [1] * 33),
    (3, 1, 64, 32, 257, [6, 3, 37, 90, 4, 3, 11, 21], [3, 3, 3, 2, 4, 3, 3, 3]),
    (8, 1, 128, 64, 384, [4, 130, 20], [4, 4, 4]),
    (1, 1, 128, 64, 260, [1 + i % 7 for i in range(97)], [1] * 97),
    (16, 2, 64, 32, 700, [1 + 9 * i for i in range(16)], [1] * 16),
    (40, 5, 128, 128, 555, [1 + 3 * i for i in range(25)], [1] * 25),
    (8, 1, 128, 256, 512, [1 + 40 * (i % 5) for i in range(32)], [1] * 32),
    (4, 1, 64, 64, 1023, [5 + i for i in range(13)], [5] * 13),
    (8, 2, 128, 32, 129, [8 + 17 * i for i in range(17)], [8, 7, 8, 8, 8, 6, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8]),
    # runs of the work split that hold whole items, two to three of them
    (16, 16, 128, 32, 140, [1 + i for i in range(34)], [1] * 34),
    (8, 8, 64, 64, 300, [1 + i % 9 for i in range(40)], [1] * 40),
    (64, 8, 128, 64, 270, [1 + 5 * (i % 6) for i in range(38)], [1] * 38),
    (32, 16, 64, 32, 140, [1 + i for i in range(36)], [1] * 36),
    (16, 8, 128, 64, 300, [1 + i % 9 for i in range(35)], [1] * 35),
    # 33 .. 64 rows with 256 an item: many heads
    (40, 40, 64, 32, 300, [1 + i % 40 for i in range(33)], [1] * 33),
])
@pytest.mark.parametrize("token", [False, True])
def test_against_the_oracle(lib, H, H_kv, d, page, prefix, own, n, token):
    """The new tokens are the last ones of each sequence."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(prefix + H)
    pair = Forked(fl, rng, prefix, own, page, H_kv, d, token=token)
    starts = [a - b for a, b in zip(pair.lens, n)]
    pair.share(n, starts)
    q, o, lse, scale = _run(fl, pair, rng, H, n, starts, prefix)
    assert pair.status.item() == 0
    _check(o, lse, pair, q, n, starts, scale)


@pytest.mark.parametrize("nseq,H,H_kv,d", [(3, 2, 2, 64), (40, 8, 2, 128), (3, 4, 1, 128)])
def test_many_tiles(lib, nseq, H, H_kv, d):
    """Prefixes of many tiles, cut between most CTAs; own tails that are cut, too."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(nseq)
    prefix = 30000 // H_kv + 5
    own = [int(rng.integers(1, 200)) for _ in range(nseq)]
    own[1] = 6001
    # (the oracle walks three sequences; the others repeat the first ones' tails)
    pair = Forked(fl, rng, prefix, own[:3], 128, H_kv, d)
    rows = [min(b, 2) if b < 3 else b % 3 for b in range(nseq)]
    pair.t = pair.t[rows]
    pair.table = torch.from_numpy(pair.t).to(DEV)
    for c in (pair.k, pair.v):
        c.codes, c.scales = [c.codes[b] for b in rows], [c.scales[b] for b in rows]
    n = [1] * nseq
    starts = [pair.lens[b] - 1 for b in rows]
    pair.share(n, starts)
    q, o, lse, scale = _run(fl, pair, rng, H, n, starts, prefix)
    assert pair.status.item() == 0
    _check(o, lse, pair, q, n, starts, scale)


@pytest.mark.parametrize("H,H_kv,d", [(4, 4, 64), (8, 1, 128), (32, 1, 128)])
def test_sequences_that_do_not_share(lib, H, H_kv, d):
    """Idle sequences, some in front; ones that stand inside the prefix, at its last token,
    at the very start or before it (no key at all); padded rows keep what they held."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(H)
    prefix = 400
    own = [3, 50, 150, 9, 3, 20, 0, 7]
    n = [0, 2, 1, 1, 2, 1, 0, 2]
    pair = Forked(fl, rng, prefix, own, 64, H_kv, d)
    starts = [0, prefix - 1, 500, 130, prefix + 1, 0, 0, -1]
    pair.share(n, starts)
    T = sum(n) + 3
    q, o, lse, scale = _run(fl, pair, rng, H, n, starts, prefix, T=T)
    assert pair.status.item() == 0
    assert (o[sum(n):] == 7).all() and (lse[:, sum(n):] == 7).all()
    _check(o[:sum(n)], lse[:, :sum(n)], pair, q, n, starts, scale)


def test_nobody_shares(lib):
    """All inside the prefix, no positions at all, or nobody there."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(2)
    pair = Forked(fl, rng, 300, [3, 5, 9], 32, 2, 64)
    n = [2, 1, 3]
    for starts in ([7, 298, 100], None):
        q = bf16(rng, (6, 8, 64)).to(DEV)
        s = None if starts is None else i32(starts)
        o, lse = pair.gpu.attend(q, offsets(n), s, pair.table, 0.1, prefix=300, dev_status=pair.status,
                                 always_share=True)
        _check(o, lse, pair, q, n, starts or [0, 0, 0], 0.1)
    o = torch.full((6, 8, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    pair.gpu.attend(q, offsets([0, 0, 0]), i32([400] * 3), pair.table, 0.1, prefix=300, o=o, dev_status=pair.status,
                     always_share=True)
    assert (o == 3).all() and pair.status.item() == 0


def test_calls_that_gain_nothing_are_the_plain_one(lib):
    """One sequence, a prefix below a tile, a window, chunks of many rows: the same bits."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(3)
    for own, n, prefix, window in (([40], [1], 300, 0), ([40, 50], [1, 1], 127, 0), ([40, 50], [1, 1], 300, 64),
                                   ([220, 250], [200, 220], 300, 0)):
        pair = Forked(fl, rng, 300, own, 64, 2, 64)
        starts = [a - b for a, b in zip(pair.lens, n)]
        q = bf16(rng, (sum(n), 4, 64)).to(DEV)
        args = q, offsets(n), i32(starts), pair.table, 0.125
        a = pair.gpu.attend(*args, window=window, sinks=4 if window else 0, prefix=prefix, always_share=True)
        b = pair.gpu.attend(*args, window=window, sinks=4 if window else 0)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("nseq,H,H_kv", [(4, 2, 1), (9, 8, 2), (33, 8, 1)])
def test_not_a_number_stays_with_those_that_see_it(lib, nseq, H, H_kv):
    """NaN in a sequence's own tail, seen by the second of its tokens only; then in a
    key of the prefix and in the unused part of the pages."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(nseq)
    prefix, d = 390, 128
    own = [2 + 3 * (b % 9) for b in range(nseq)]
    n, pair = [2] * nseq, None
    pair = Forked(fl, rng, prefix, own, 64, H_kv, d)
    starts = [x - 2 for x in pair.lens]
    last = pair.lens[1] - 1
    page = int(pair.t[1, last // 64])
    pair.share(n, starts)
    q, want, lse, scale = _run(fl, pair, rng, H, n, starts, prefix)
    pair.gpu.v_codes[page, 0, last % 64, 5] = 0x7F
    _, o, _, _ = _run(fl, pair, rng, H, n, starts, prefix, q=q)
    G = H // H_kv
    # (a value that not all rows see moves its NaN into the weights of those that do)
    assert torch.isnan(o[3, :G, 5]).all()
    o[3, :G] = 0
    assert not torch.isnan(o).any()
    pair.gpu.v_codes[page, 0, last % 64, 5] = 0
    pair.gpu.k_codes[int(pair.t[0, 1]), 0, 3] = 0x7F
    _, o, lse, _ = _run(fl, pair, rng, H, n, starts, prefix, q=q)
    assert torch.isnan(o[:, :G]).all() and not torch.isnan(o[:, G:]).any()
    assert torch.isnan(lse[:G]).all() and not torch.isnan(lse[G:]).any()


@pytest.mark.parametrize("scale", [1e-30, 3.0, 3e4])
def test_flat_and_steep_softmax(lib, scale):
    """Scores all alike; far apart; beyond 2^16, where the prefix or the tail wins alone."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(4)
    for nseq in (3, 30):
        pair = Forked(fl, rng, 270, [1 + 5 * b for b in range(nseq)], 32, 1, 64)
        n = [1] * nseq
        starts = [x - 1 for x in pair.lens]
        pair.share(n, starts)
        q, o, lse, _ = _run(fl, pair, rng, 4, n, starts, 270, scale=scale)
        if scale < 1e3:
            _check(o, lse, pair, q, n, starts, scale)
            continue
        for b in range(nseq):  # a mean of values whose scores come within the stated 2^-19
            for h in range(4):
                x = pair.k.values(b)[:, 0] @ q[b, h].double().cpu().numpy() * scale
                near = x >= x.max() - 2.0 ** -18 * np.abs(x).max() - 40
                v = pair.v.values(b)[near, 0]
                got = o[b, h].double().cpu().numpy()
                slack = 2.0 ** -7 * np.abs(v).max() + 2.0 ** -24 * np.abs(pair.v.values(b)).max() * len(x)
                assert (got >= v.min(0) - slack).all() and (got <= v.max(0) + slack).all()


def test_runs_repeat_and_streams_and_graphs_agree(lib):
    """The same bits in every run, on two streams at once, captured and replayed."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(5)
    nseq, H, H_kv, d, prefix = 48, 16, 4, 128, 3001
    pair = Forked(fl, rng, prefix, [1 + 11 * b for b in range(nseq)], 64, H_kv, d)
    n = [1] * nseq
    starts = [x - 1 for x in pair.lens]
    pair.share(n, starts)
    q = [bf16(rng, (nseq, H, d)).to(DEV) for _ in range(2)]
    cu, st = offsets(n), i32(starts)
    args = cu, st, pair.table, d ** -0.5
    want = [pair.gpu.attend(x, *args, prefix=prefix, always_share=True) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(pair.gpu.attend(q[i], *args, prefix=prefix, always_share=True))
    graphs, outs = [], []
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(pair.gpu.attend(q[i], *args, prefix=prefix, always_share=True))
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i] + [outs[i]]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    # strided queries, no lse, a workspace of the caller's
    big = torch.zeros(nseq, H + 2, d, dtype=torch.bfloat16, device=DEV)
    big[:, 1:H + 1] = q[0]
    ws = torch.empty(fl.flamia_attn_cache_prefix_workspace_bytes(nseq, nseq, H, H_kv, d, prefix, fl.FLAG_PREFIX_ALWAYS),
                     dtype=torch.uint8, device=DEV)
    o = torch.empty_like(q[0])
    fl.flamia_attn_cache_prefix(pair.gpu, big[:, 1:H + 1], cu, st, pair.table, prefix, d ** -0.5, o, None, ws,
                                pair.status, fl.FLAG_PREFIX_ALWAYS)
    assert torch.equal(o, want[0][0]) and pair.status.item() == 0


def test_pages_outside_the_pool_are_reported(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(6)
    for nseq in (3, 30):
        pair = Forked(fl, rng, 300, [20] * nseq, 64, 1, 64)
        n, starts = [1] * nseq, [319] * nseq
        pair.share(n, starts)
        pair.table[0, 1] = pair.gpu.num_pages
        _run(fl, pair, rng, 4, n, starts, 300)
        assert pair.status.item() == fl.DEV_BAD_PAGE
        pair.status.zero_()
        _run(fl, pair, rng, 4, n, [319] * (nseq - 1) + [100000], 300)  # outside its row
        assert pair.status.item() == fl.DEV_BAD_PAGE


def test_more_sequences_than_threads(lib):
    """The plan walks several sequences a thread."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(7)
    nseq, prefix = 1100, 129
    pair = Forked(fl, rng, prefix, [4, 40, 9], 32, 1, 64)
    rows = [b % 3 for b in range(nseq)]
    pair.t = pair.t[rows]
    pair.table = torch.from_numpy(pair.t).to(DEV)
    for c in (pair.k, pair.v):
        c.codes, c.scales = [c.codes[b] for b in rows], [c.scales[b] for b in rows]
    n = [0 if b < 5 or b % 4 == 2 else 1 for b in range(nseq)]
    starts = [pair.lens[b] - 1 if i % 7 else 60 for i, b in enumerate(rows)]
    q, o, lse, scale = _run(fl, pair, rng, 2, n, starts, prefix)
    assert pair.status.item() == 0
    _check(o, lse, pair, q, n, starts, scale)


@pytest.mark.parametrize("nseq,H", [(5, 2), (30, 8)])
def test_a_sequence_outside_its_row_spoils_no_other(lib, nseq, H):
    """The first sequence stands behind its table row: it is reported, and the pages of the
    next one are read for the others."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(8)
    prefix = 300
    pair = Forked(fl, rng, prefix, [5 + b for b in range(nseq)], 64, 1, 64)
    n, starts = [1] * nseq, [x - 1 for x in pair.lens]
    pair.share([0] + n[1:], starts)
    pair.table[0] = -1
    starts[0] = 64 * pair.t.shape[1]
    q, o, lse, scale = _run(fl, pair, rng, H, n, starts, prefix)
    assert pair.status.item() == fl.DEV_BAD_PAGE
    for b in range(1, nseq):
        k, v = pair.k.values(b), pair.v.values(b)
        ref, _ = S.attend(q[b:b + 1].double().cpu().numpy(), k, v, starts[b], scale)
        assert np.abs(o[b:b + 1].double().cpu().numpy() - ref).max() <= 2.0 ** -7 * np.abs(v).max()


@pytest.mark.parametrize("nseq,H", [(5, 2), (5, 8), (7, 16)])
def test_rows_of_no_sequence(lib, nseq, H):
    """Offsets that begin behind the first rows are reported; whatever the workspace held for
    those rows, the others' results are right."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(nseq + H)
    prefix, own, H_kv, d = 300, [3 + 40 * b for b in range(nseq)], 1, 64
    pair = Forked(fl, rng, prefix, own, 64, H_kv, d)
    n, gap = [1] * nseq, 3
    starts = [x - 1 for x in pair.lens]
    pair.share(n, starts)
    T = nseq + gap
    q = bf16(rng, (T, H, d)).to(DEV)
    o, lse = (torch.full(s, 7.0, dtype=t, device=DEV)
              for s, t in (((T, H, d), torch.bfloat16), ((H, T), torch.float32)))
    size = fl.flamia_attn_cache_prefix_workspace_bytes(T, nseq, H, H_kv, d, prefix,
                                                       fl.FLAG_PREFIX_ALWAYS)
    # records of parts beyond the last CTA of 256 rows an item; then of no CTA at all
    for at, parts in ((320, 100 | 1 << 30), (511, 1 << 30 | 1), (-1, -1)):
        ws = i32([at, parts]).repeat((size + 7) // 8).view(torch.uint8)[:size]
        pair.status.zero_()
        pair.gpu.attend(q, offsets(n) + gap, i32(starts), pair.table, d ** -0.5, prefix=prefix, o=o,
                        lse=lse, ws=ws, dev_status=pair.status, always_share=True)
        assert pair.status.item() == 1
        _check(o[gap:], lse[:, gap:], pair, q[gap:], n, starts, d ** -0.5)
