"""Attention over the paged cache with many query rows a sequence and K / V head
(more than 96 on average: items of 256 rows), against float64 attention."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, Pair, bf16, check_attend, i32, offsets
from tests.test_gpu_attn_cache import RAMPS, _ramp, _run, test_many_tiles_a_cta as many_tiles

pytestmark = pytest.mark.gpu


def _rows(n, H, H_kv):
    """Mean rows a sequence and K / V head: the kernel's rule."""
    rows = -(-sum(n) // len(n)) * (H // H_kv)
    assert rows > 96, rows


SHAPES = [
    # new tokens, contexts before them, H, H_kv, d, page
    ([145], [0], 1, 1, 64, 32),
    ([200], [0], 1, 1, 128, 64),
    ([135], [5], 1, 1, 128, 32),
    ([129], [127], 1, 1, 64, 128),
    ([130], [0], 2, 1, 64, 128),
    ([256], [128], 2, 2, 128, 256),
    ([257], [100], 1, 1, 128, 384),
    ([300, 1, 0, 77], [10, 600, 50, 0], 8, 2, 64, 64),
    ([300, 1, 0, 77], [10, 600, 50, 0], 4, 2, 128, 32),
    ([9, 12], [400, 3], 35, 1, 64, 32),
    ([70, 90, 200], [60, 300, 0], 6, 3, 128, 64),
    ([17, 3], [250, 1111], 16, 1, 128, 128),
    ([513, 255, 256], [700, 1, 0], 3, 3, 64, 32),
]


@pytest.mark.parametrize("n,starts,H,H_kv,d,page", SHAPES)
@pytest.mark.parametrize("token", [False, True])
def test_chunks(lib, n, starts, H, H_kv, d, page, token):
    from precision_causal_attention_block_gb300 import flamia as fl
    _rows(n, H, H_kv)
    _run(fl, np.random.default_rng(sum(n) + d), n, starts, H, H_kv, d, page, token=token)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (32, 0), (100, 130), (128, 4),
                                          (129, 64), (300, 1), (5000, 3)])
def test_window_and_first_tokens(lib, window, sinks):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(window + sinks)
    for n, starts, H, H_kv, d, page in (([170, 4, 1, 140], [700, 383, 0, 250], 4, 2, 64, 32),
                                        ([270, 30], [511, 900], 2, 1, 128, 128)):
        _rows(n, H, H_kv)
        _run(fl, rng, n, starts, H, H_kv, d, page, window=window, sinks=sinks)


def test_magnitudes_and_positions_that_see_nothing(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(51)
    for token in (False, True):
        _run(fl, rng, [100, 90], [300, 90], 4, 2, 128, 64, token, q_scale=12.0)
        _run(fl, rng, [100], [300], 4, 2, 64, 64, token, q_scale=1e-3, k_scale=1e3, v_scale=1e-20)
        _run(fl, rng, [100], [90], 4, 2, 64, 64, token, q_scale=1e18, k_scale=1e-18, v_scale=1e25)
    _run(fl, rng, [150, 100, 200], [-30, -100, 10], 4, 2, 64, 32)


@pytest.mark.parametrize("token", [False, True])
def test_first_token_of_zero_value_takes_the_weight(lib, token):
    """As for single tokens: its block of 32 has the lowest exponent."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(52)
    n, L, H_kv = 150, 400, 2
    for top in (10.0, 40.0, 95.0):
        for d in (64, 128):
            pair = Pair(fl, rng, [L], 64, H_kv, d, token)
            q = torch.zeros(n, H_kv, d, dtype=torch.bfloat16)
            q[..., 0] = d ** 0.5
            k, v = bf16(rng, (L, H_kv, d)), bf16(rng, (L, H_kv, d))
            k[0, :, 0] = top
            v[:32] = 0
            pair.write(k, v, [L], [0])
            q = q.to(DEV)
            o, lse = pair.gpu.attend(q, offsets([n]), i32([L - n]), pair.table, d ** -0.5)
            check_attend(o, lse, pair, q, [n], [L - n], d ** -0.5)


@pytest.mark.parametrize("name", sorted(RAMPS))
@pytest.mark.parametrize("n,H,H_kv,d,token", [(140, 2, 2, 128, False), (70, 4, 2, 64, False),
                                              (260, 1, 1, 64, True)])
def test_changing_magnitudes_along_a_sequence(lib, name, n, H, H_kv, d, token):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(len(name) + n)
    L, nseq = 1230, 60
    pair = Pair(fl, rng, [L], 64, H_kv, d, token)
    k, v = _ramp(rng, L, H_kv, d, *RAMPS[name])
    pair.write(k, v, [L], [0])
    table = pair.table.expand(nseq, -1).contiguous()  # the same pages in every sequence
    q1 = bf16(rng, (n, H, d))
    q = q1.repeat(nseq, 1, 1).to(DEV)
    o, lse = pair.gpu.attend(q, offsets([n] * nseq), i32([L - n] * nseq), table, d ** -0.5)
    check_attend(o[:n], lse[:, :n].contiguous(), pair, q[:n], [n], [L - n], d ** -0.5)
    far = (o.view(nseq, n, H, d).float() - o[:n].float()).abs().max()
    assert float(far) <= 2.0 ** -6 * float(o[:n].float().abs().max())


def test_nan_stays_where_it_is_seen(lib):
    """NaN keys and values that some rows of an item see and others do not, and NaN
    queries: rows that meet none are the same without them."""
    from precision_causal_attention_block_gb300 import flamia as fl
    n, H, H_kv, L = 180, 4, 2, 520
    for d, which in ((64, "k"), (64, "v"), (128, "k"), (128, "v")):
        outs = []
        for plant in (True, False):
            rng = np.random.default_rng(53)
            pair = Pair(fl, rng, [L, L], 32, H_kv, d)
            k, v = bf16(rng, (2 * L, H_kv, d)), bf16(rng, (2 * L, H_kv, d))
            q = bf16(rng, (2 * n, H, d))
            if plant:
                x = k if which == "k" else v
                x[100, :, 3] = float("nan")       # sequence 0: behind every window
                x[L + 500, 0, 5] = float("inf")   # sequence 1: rows 160 .. of head 0's group
                x[L + 260, 1, 0] = float("nan")   # rows up to 69 of head 1's group
                q[7, 1, 5] = float("nan")
            pair.write(k, v, [L, L], [0, 0])
            outs.append(pair.gpu.attend(q.to(DEV), offsets([n, n]), i32([L - n] * 2), pair.table,
                                        d ** -0.5, window=150)[0])
            if not plant:
                o, lse = pair.gpu.attend(q.to(DEV), offsets([n, n]), i32([L - n] * 2), pair.table,
                                         d ** -0.5, window=150)
                check_attend(o, lse, pair, q.to(DEV), [n, n], [L - n] * 2, d ** -0.5, 150)
        bad = torch.isnan(outs[0]).cpu().numpy()
        want = np.zeros((2 * n, H), dtype=bool)
        want[7, 1] = True
        want[n + 160:, :2] = True
        want[n:n + 70, 2:] = True
        assert np.array_equal(bad.any(-1), want), (d, which)
        got, ref = outs[0].double().cpu().numpy()[~want], outs[1].double().cpu().numpy()[~want]
        # (a block's exponent may differ where a planted element was its largest)
        assert np.abs(got - ref).max() <= 2.0 ** -6 * np.abs(ref).max()


def test_repeatable_padded_and_captured(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(54)
    n, starts, H, H_kv, d = [300, 0, 200, 0], [1000, 7, 1300, 0], 4, 2, 128
    pair, q, o, lse = _run(fl, rng, n, starts, H, H_kv, d, 64)
    T = sum(n) + 3
    wide = torch.zeros(T, 2 * H, d, dtype=torch.bfloat16, device=DEV)
    wide[:sum(n), H:] = q
    o2 = torch.full((T, H, d), 3.0, dtype=torch.bfloat16, device=DEV)
    lse2 = torch.full((H, T), 5.0, device=DEV)
    cu, st = offsets(n), i32(starts)
    run = lambda: pair.gpu.attend(wide[:, H:], cu, st, pair.table, d ** -0.5, o=o2, lse=lse2)
    run()
    assert torch.equal(o2[:sum(n)], o) and torch.equal(lse2[:, :sum(n)], lse)
    assert bool((o2[sum(n):] == 3.0).all()) and bool((lse2[:, sum(n):] == 5.0).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            run()
    o2.zero_()
    g.replay()
    assert torch.equal(o2[:sum(n)], o)
    # single tokens of the same cache between two chunks
    one = bf16(rng, (4, H, d)).to(DEV)
    last = i32([1299, 6, 1499, 0])
    table, a1 = pair.table, offsets([1, 0, 1, 0])
    w1, _ = pair.gpu.attend(one[:2], a1, last, table, d ** -0.5)
    for _ in range(5):
        run()
        w2, _ = pair.gpu.attend(one[:2], a1, last, table, d ** -0.5)
        assert torch.equal(w1, w2)
    assert torch.equal(o2[:sum(n)], o)


def test_bad_pages_are_reported(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(55)
    n, L, H, d = 140, 700, 2, 64
    pair = Pair(fl, rng, [L, L], 32, H, d)
    pair.write(bf16(rng, (2 * L, H, d)), bf16(rng, (2 * L, H, d)), [L, L], [0, 0])
    q = bf16(rng, (2 * n, H, d)).to(DEV)
    cu = offsets([n, n])
    good, _ = pair.gpu.attend(q, cu, i32([L - n] * 2), pair.table, 0.125)
    for entry in (-1, pair.gpu.num_pages, 1 << 30, -(1 << 31)):
        bad = pair.table.clone()
        bad[1, 2] = entry
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o, _ = pair.gpu.attend(q, cu, i32([L - n] * 2), bad, 0.125, dev_status=st)
        assert int(st.item()) == fl.DEV_BAD_PAGE
        assert torch.equal(o[:n], good[:n]) and bool(torch.isfinite(o.float()).all())
        st.zero_()
        pair.gpu.attend(q, cu, i32([L - n] * 2), bad, 0.125, window=3, dev_status=st)
        assert int(st.item()) == 0
    for start in (L, 1 << 29, (1 << 30) - n, 1 << 30, (1 << 31) - 1):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o, _ = pair.gpu.attend(q, cu, i32([L - n, start]), pair.table, 0.125, dev_status=st)
        assert int(st.item()) == fl.DEV_BAD_PAGE, start
        # (other parts of the work may be cut elsewhere)
        assert float((o[:n].float() - good[:n].float()).abs().max()) <= 2.0 ** -7 * float(
            good[:n].float().abs().max()), start
    for off in ([0, n, 3 * n], [0, 2 * n, n], [1, n, 2 * n]):
        st.zero_()
        pair.gpu.attend(q, i32(off), i32([L - n] * 2), pair.table, 0.125, dev_status=st)
        assert int(st.item()) & fl.DEV_BAD_SEQLENS, off


LONG_RUNS = [
    # sequences, longest context, new tokens, H, H_kv, d, page, window, sinks
    (30, 2500, 400, 8, 8, 64, 32, 0, 0),
    (12, 6000, 700, 4, 2, 128, 64, 0, 0),
    (20, 4000, 200, 8, 2, 128, 256, 900, 130),
    (9, 5000, 900, 12, 3, 64, 128, 2000, 4),
]


@pytest.mark.parametrize("nseq,longest,new,H,H_kv,d,page,window,sinks", LONG_RUNS)
def test_many_tiles_a_cta(lib, nseq, longest, new, H, H_kv, d, page, window, sinks):
    many_tiles(lib, nseq, longest, new, H, H_kv, d, page, window, sinks)
