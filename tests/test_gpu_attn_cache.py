"""Attention over the paged cache against float64 attention of the cached values."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, Pair, bf16, check_attend, i32, offsets

pytestmark = pytest.mark.gpu


def _run(fl, rng, n, starts, H, H_kv, d, page, token=False, window=0, sinks=0, q_scale=1.0,
         k_scale=1.0, v_scale=1.0, width=None):
    lens = [max(s, 0) + c for s, c in zip(starts, n)]
    pair = Pair(fl, rng, lens, page, H_kv, d, token, width=width)
    if sum(lens):
        pair.write(bf16(rng, (sum(lens), H_kv, d), k_scale), bf16(rng, (sum(lens), H_kv, d), v_scale),
                   lens, [0] * len(n))
    T = sum(n)
    q = bf16(rng, (T, H, d), q_scale).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = pair.gpu.attend(q, offsets(n), i32(starts), pair.table, d ** -0.5, window=window,
                             sinks=sinks, dev_status=st)
    assert int(st.item()) == 0
    check_attend(o, lse, pair, q, n, starts, d ** -0.5, window, sinks)
    return pair, q, o, lse


SINGLE = [
    # contexts before the token, H, H_kv, d, page
    ([0], 1, 1, 64, 32),
    ([0, 1, 31, 32, 33], 2, 2, 64, 32),
    ([126, 127, 128, 129], 4, 2, 128, 64),
    ([300, 0, 1000, 511], 8, 1, 128, 128),
    ([63, 255, 257], 7, 1, 64, 64),
    ([640, 100], 16, 1, 128, 256),
    ([77, 400], 20, 1, 64, 32),
    ([1500], 3, 3, 128, 32),
    ([1023], 5, 5, 64, 384),
]


@pytest.mark.parametrize("ctx,H,H_kv,d,page", SINGLE)
@pytest.mark.parametrize("token", [False, True])
def test_single_tokens(lib, ctx, H, H_kv, d, page, token):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(len(ctx) + H + d + page)
    _run(fl, rng, [1] * len(ctx), ctx, H, H_kv, d, page, token)


SEVERAL = [
    # new tokens, contexts before them, H, H_kv, d, page
    ([1, 4, 0, 2], [10, 200, 50, 0], 4, 2, 128, 32),
    ([3, 9, 1], [125, 127, 700], 4, 4, 64, 64),
    ([130], [0], 2, 1, 64, 128),
    ([70, 1, 33], [60, 300, 0], 6, 3, 128, 64),
    ([257], [100], 1, 1, 128, 32),
    ([5, 5], [400, 3], 35, 5, 64, 32),
    ([17], [250], 16, 1, 128, 128),
]


@pytest.mark.parametrize("n,starts,H,H_kv,d,page", SEVERAL)
def test_several_tokens(lib, n, starts, H, H_kv, d, page):
    from precision_causal_attention_block_gb300 import flamia as fl
    _run(fl, np.random.default_rng(sum(n) + d), n, starts, H, H_kv, d, page)


WINDOWS = [(1, 0), (1, 1), (7, 4), (32, 0), (100, 130), (128, 4), (129, 64), (300, 1), (5000, 3)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_and_first_tokens(lib, window, sinks):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(window + sinks)
    _run(fl, rng, [1, 4, 1, 40], [700, 383, 0, 250], 4, 2, 64, 32, window=window, sinks=sinks)
    _run(fl, rng, [1, 3], [511, 90], 8, 1, 128, 128, window=window, sinks=sinks)


def test_magnitudes(lib):
    """Peaked softmax, tiny and huge values, blocks of very different exponents."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(21)
    _run(fl, rng, [2, 1], [300, 90], 4, 2, 128, 64, q_scale=12.0)
    _run(fl, rng, [1, 1], [300, 90], 4, 2, 64, 64, q_scale=1e-3, k_scale=1e3, v_scale=1e-20)
    _run(fl, rng, [1, 1], [300, 90], 4, 2, 64, 64, q_scale=1e18, k_scale=1e-18, v_scale=1e25)


def test_first_token_of_zero_value_takes_the_weight(lib):
    """A key whose score tops the rest by 40 nats and whose value is zero (its block
    of 32 has the lowest exponent): the output is what the others leave."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(22)
    for top in (10.0, 40.0, 95.0):
        for d in (64, 128):
            H_kv, L = 2, 400
            pair = Pair(fl, rng, [L], 64, H_kv, d)
            q = torch.zeros(1, H_kv, d, dtype=torch.bfloat16)
            q[..., 0] = d ** 0.5
            k, v = bf16(rng, (L, H_kv, d)), bf16(rng, (L, H_kv, d))
            k[0, :, 0] = top
            v[:32] = 0
            pair.write(k, v, [L], [0])
            q = q.to(DEV)
            o, lse = pair.gpu.attend(q, offsets([1]), i32([L - 1]), pair.table, d ** -0.5)
            check_attend(o, lse, pair, q, [1], [L - 1], d ** -0.5)


def _ramp(rng, L, H_kv, d, k_of, v_of):
    k, v = bf16(rng, (L, H_kv, d)).double(), bf16(rng, (L, H_kv, d)).double()
    p = torch.arange(L, dtype=torch.float64)[:, None, None]
    return (k * k_of(p)).to(torch.bfloat16), (v * v_of(p)).to(torch.bfloat16)


RAMPS = {
    # keys that grow along the sequence: the references move again and again
    "growing keys": (lambda p: 0.05 + p / 120, lambda p: 1.0 + 0 * p),
    "shrinking keys": (lambda p: 12 - p / 120, lambda p: 1.0 + 0 * p),
    # values whose exponents climb or fall by more than their references' range
    "climbing values": (lambda p: 1.0 + 0 * p, lambda p: 10.0 ** (-30 + p / 20)),
    "falling values": (lambda p: 1.0 + 0 * p, lambda p: 10.0 ** (30 - p / 20)),
    "a step up": (lambda p: 1.0 + 0 * p, lambda p: torch.where(p < 700, 1e-25, 1e12)),
    "a step down": (lambda p: 1.0 + 0 * p, lambda p: torch.where(p < 700, 1e12, 1e-25)),
}


@pytest.mark.parametrize("name", sorted(RAMPS))
@pytest.mark.parametrize("n,H,H_kv,d", [(1, 2, 2, 128), (1, 2, 1, 64), (6, 4, 2, 128),
                                        (40, 2, 2, 64)])
def test_changing_magnitudes_along_a_sequence(lib, name, n, H, H_kv, d):
    """Several tiles an item (many sequences share the CTAs), scores or value
    exponents that change by far more than the slack of the running references."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(len(name) + n)
    L, nseq = 1230, 150
    pair = Pair(fl, rng, [L], 64, H_kv, d)
    k, v = _ramp(rng, L, H_kv, d, *RAMPS[name])
    pair.write(k, v, [L], [0])
    table = pair.table.expand(nseq, -1).contiguous()  # the same pages in every sequence
    q1 = bf16(rng, (n, H, d))
    q = q1.repeat(nseq, 1, 1).to(DEV)
    o, lse = pair.gpu.attend(q, offsets([n] * nseq), i32([L - n] * nseq), table, d ** -0.5)
    # the same sequence everywhere; cut into parts at different places
    check_attend(o[:n], lse[:, :n].contiguous(), pair, q[:n], [n], [L - n], d ** -0.5)
    far = (o.view(nseq, n, H, d).float() - o[:n].float()).abs().max()
    assert float(far) <= 2.0 ** -6 * float(o[:n].float().abs().max())


def test_nan_and_infinite_queries_touch_their_row_only(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(41)
    for n, H in ((1, 4), (3, 4), (9, 4)):
        pair = Pair(fl, rng, [300, 300], 64, 2, 64)
        pair.write(bf16(rng, (600, 2, 64)), bf16(rng, (600, 2, 64)), [300, 300], [0, 0])
        q = bf16(rng, (2 * n, H, 64)).to(DEV)
        args = (offsets([n, n]), i32([300 - n] * 2), pair.table, 0.125)
        good, _ = pair.gpu.attend(q, *args)
        q[0, 1, 5] = float("nan")
        q[n, 3, 0] = float("-inf")
        bad, _ = pair.gpu.attend(q, *args)
        hit = torch.zeros(2 * n, H, dtype=torch.bool, device=DEV)
        hit[0, 1] = hit[n, 3] = True
        assert bool(torch.isnan(bad[hit]).all()) and torch.equal(bad[~hit], good[~hit])


def test_workspace_of_a_cache_never_moves(lib):
    """A captured call stays valid when later calls have more rows an item."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(42)
    pair = Pair(fl, rng, [900] * 4, 64, 1, 64)
    pair.write(bf16(rng, (3600, 1, 64)), bf16(rng, (3600, 1, 64)), [900] * 4, [0] * 4)
    q = bf16(rng, (4, 1, 64)).to(DEV)
    cu, st = offsets([1] * 4), i32([899] * 4)
    o, lse = torch.zeros_like(q), torch.zeros(1, 4, device=DEV)
    run = lambda: pair.gpu.attend(q, cu, st, pair.table, 0.125, o=o, lse=lse)
    run()
    want = o.clone()
    at = pair.gpu._ws.data_ptr()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    big = bf16(rng, (160, 8, 64)).to(DEV)
    pair.gpu.attend(big, offsets([40] * 4), i32([860] * 4), pair.table, 0.125)
    assert pair.gpu._ws.data_ptr() == at
    o.zero_()
    g.replay()
    assert torch.equal(o, want)


def test_no_tokens(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    c = fl.KVCache(2, 32, 1, 64)
    z = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    t = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    cu = i32([0, 0, 0])
    before = lib.flamia_debug_launch_count()
    c.write(z, z, cu, None, t)
    k, _ = c.read(cu, None, t, 0)
    o, lse = c.attend(z, cu, None, t, 0.125)
    fl.Rotary(fl.rope_frequencies(64))(z, z, cu)
    assert k.shape == (0, 1, 64) and o.shape == (0, 1, 64) and lse.shape == (1, 0)
    assert lib.flamia_debug_launch_count() == before
    # and sequences that are all idle in a padded batch
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    o = torch.full_like(x, 5.0)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.write(x, x, cu, None, t, dev_status=st)
    c.attend(x, cu, None, t, 0.125, o=o, dev_status=st)
    assert bool((o == 5.0).all()) and not bool(c.k_codes.any()) and int(st.item()) == 0


def test_nan_stays_where_it_is_seen(lib):
    """NaN keys and values outside the window, behind the end or in other
    sequences change nothing; a query that sees one gives NaN, its neighbours do not."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(23)
    for d, which in ((64, "k"), (64, "v"), (128, "k"), (128, "v")):
        H, L, n = 4, 300, 20
        pair = Pair(fl, rng, [L, L], 32, 2, d)
        k, v = bf16(rng, (2 * L, 2, d)), bf16(rng, (2 * L, 2, d))
        bad = k if which == "k" else v
        bad[100, :, 3] = float("nan")      # sequence 0, position 100
        bad[L + 290, 0, 5] = float("inf")  # sequence 1, position 290, head 0
        pair.write(k, v, [L, L], [0, 0])
        q = bf16(rng, (2 * n, H, d)).to(DEV)
        o, _ = pair.gpu.attend(q, offsets([n, n]), i32([L - n] * 2), pair.table, d ** -0.5,
                                 window=150)
        # sequence 0: queries 280 .. 299 see keys from 131 on
        one = torch.isnan(o).cpu().numpy().any(-1)
        assert not one[:n].any()
        want = np.zeros((n, H), dtype=bool)
        want[10:, :2] = True
        assert np.array_equal(one[n:], want)
        # without the NaN the clean rows are the same
        bad[100, :, 3] = 0
        bad[L + 290, 0, 5] = 0
        pair2 = Pair(fl, np.random.default_rng(23), [L, L], 32, 2, d)
        pair2.write(k, v, [L, L], [0, 0])
        o2, lse2 = pair2.gpu.attend(q, offsets([n, n]), i32([L - n] * 2), pair2.table, d ** -0.5,
                                    window=150)
        check_attend(o2, lse2, pair2, q, [n, n], [L - n] * 2, d ** -0.5, 150)
        got, ref = o.double().cpu().numpy(), o2.double().cpu().numpy()
        clean = ~np.isnan(got)
        # two BF16 roundings of values that the tolerance of check_attend holds apart
        assert np.abs(got[clean] - ref[clean]).max() <= 2.0 ** -6 * np.abs(ref).max()


def test_rows_that_see_nothing(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(24)
    _run(fl, rng, [5, 1, 3], [-3, -1, 10], 4, 2, 64, 32)


def test_padded_batch_and_rows_behind_it(lib):
    """Idle sequences between and behind the others; rows and columns behind the
    last token keep their bits."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(25)
    n, starts, H, d = [1, 0, 2, 0, 0], [40, 7, 130, 0, 0], 4, 128
    pair = Pair(fl, rng, [s + c for s, c in zip(starts, n)], 64, 2, d)
    lens = [s + c for s, c in zip(starts, n)]
    pair.write(bf16(rng, (sum(lens), 2, d)), bf16(rng, (sum(lens), 2, d)), lens, [0] * 5)
    T = 6
    q = bf16(rng, (T, H, d)).to(DEV)
    o = torch.full((T, H, d), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((H, T), 5.0, device=DEV)
    pair.gpu.attend(q, offsets(n), i32(starts), pair.table, d ** -0.5, o=o, lse=lse)
    assert bool((o[3:] == 3.0).all()) and bool((lse[:, 3:] == 5.0).all())
    check_attend(o[:3], lse[:, :3].contiguous(), pair, q[:3], n, starts, d ** -0.5)
    # without lse, and from a strided q
    wide = torch.zeros(T, 2 * H, d, dtype=torch.bfloat16, device=DEV)
    wide[:, H:] = q
    o2 = torch.zeros_like(o)
    ws = torch.empty(fl.flamia_attn_cache_workspace_bytes(T, 5, H, 2, d), dtype=torch.uint8, device=DEV)
    fl.flamia_attn_cache(pair.gpu, wide[:, H:], offsets(n), i32(starts), pair.table, d ** -0.5, 0,
                         0, o2, None, ws)
    assert torch.equal(o2[:3], o[:3])


def test_shared_pages(lib):
    """Two sequences over the same pages (a shared prompt)."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(26)
    pair = Pair(fl, rng, [200], 64, 2, 64)
    pair.write(bf16(rng, (200, 2, 64)), bf16(rng, (200, 2, 64)), [200], [0])
    q = bf16(rng, (1, 4, 64)).to(DEV)
    o, _ = pair.gpu.attend(q, offsets([1]), i32([199]), pair.table, 0.125)
    two = torch.cat([pair.table, pair.table])
    o2, _ = pair.gpu.attend(torch.cat([q, q]), offsets([1, 1]), i32([199, 199]), two, 0.125)
    assert torch.equal(o2[0], o2[1])
    assert (o2[0].float() - o[0].float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()


def test_bad_pages_are_reported(lib):
    """Bad entries that the call needs are reported; entries that it does not need
    are not looked at; the other sequences are served."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(27)
    n, starts = [1, 1], [99, 99]
    pair = Pair(fl, rng, [100, 100], 32, 2, 64)
    x, y = bf16(rng, (200, 2, 64)), bf16(rng, (200, 2, 64))
    pair.write(x, y, [100, 100], [0, 0])
    q = bf16(rng, (2, 2, 64)).to(DEV)
    good, _ = pair.gpu.attend(q, offsets(n), i32(starts), pair.table, 0.125)
    for entry in (-1, pair.gpu.num_pages, 1 << 30, -(1 << 31)):
        bad = pair.table.clone()
        bad[1, 2] = entry
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o, _ = pair.gpu.attend(q, offsets(n), i32(starts), bad, 0.125, dev_status=st)
        assert int(st.item()) == fl.DEV_BAD_PAGE
        assert torch.equal(o[0], good[0])
        # a window that does not reach the bad page
        st.zero_()
        pair.gpu.attend(q, offsets(n), i32(starts), bad, 0.125, window=3, dev_status=st)
        assert int(st.item()) == 0
    # positions outside the table
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, _ = pair.gpu.attend(q, offsets(n), i32([99, 128]), pair.table, 0.125, dev_status=st)
    assert int(st.item()) == fl.DEV_BAD_PAGE and torch.equal(o[0], good[0])
    for cu in ([0, 1, 3], [0, 2, 1], [1, 1, 2]):
        st.zero_()
        pair.gpu.attend(q, i32(cu), i32([99, 99]), pair.table, 0.125, dev_status=st)
        assert int(st.item()) & fl.DEV_BAD_SEQLENS, cu


@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 0), (70, 1 << 29)])
@pytest.mark.parametrize("pages", [4, 40])
def test_first_positions_far_outside_the_table(lib, window, sinks, pages):
    """They are reported, the walk over keys ends with the page table (a walk to the
    position would be 2^22 tiles, seconds), and the other sequence is served."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(33)
    pair = Pair(fl, rng, [128, 128], 32, 2, 64)
    pair.write(bf16(rng, (256, 2, 64)), bf16(rng, (256, 2, 64)), [128, 128], [0, 0])
    table = torch.zeros(2, pages, dtype=torch.int32, device=DEV)
    table[:, :4] = pair.table
    table[1, 4:] = pair.table[1, 0]
    q = bf16(rng, (2, 2, 64)).to(DEV)
    cu = offsets([1, 1])
    good, _ = pair.gpu.attend(q, cu, i32([127, 127]), table, 0.125, window, sinks)
    for start in (1 << 29, (1 << 30) - 1, 1 << 30, (1 << 31) - 1):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        starts = i32([127, start])
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        o, _ = pair.gpu.attend(q, cu, starts, table, 0.125, window, sinks, dev_status=st)
        end.record()
        torch.cuda.synchronize()
        assert int(st.item()) == fl.DEV_BAD_PAGE, start
        assert torch.equal(o[0], good[0]) and bool(torch.isfinite(o[1].float()).all()), start
        assert begin.elapsed_time(end) < 500.0, start


def test_repeatable_and_two_streams(lib):
    """The same call twice gives the same bits; two calls at once on two streams, a
    workspace each, too."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(28)
    n, starts, H, d = [1] * 6, [5, 900, 2000, 64, 300, 1999], 8, 128
    pair, q, o, lse = _run(fl, rng, n, starts, H, 2, d, 64)
    cu, st = offsets(n), i32(starts)
    outs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ws = torch.empty(fl.flamia_attn_cache_workspace_bytes(6, 6, H, 2, d), dtype=torch.uint8,
                         device=DEV)
        with torch.cuda.stream(s):
            for _ in range(20):
                got = pair.gpu.attend(q, cu, st, pair.table, d ** -0.5, ws=ws)
            outs.append((s, got, ws))
    for s, got, _ in outs:
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)


def test_rows_beyond_32_bits_of_a_large_cache(lib):
    """Pages whose codes lie more than 2^32 bytes into the pool."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(29)
    pages, page, H_kv, d = 70000, 256, 2, 128  # 4.6e9 bytes each of K and V
    c = fl.KVCache(pages, page, H_kv, d)
    small = fl.KVCache(8, page, H_kv, d)
    far = torch.tensor([[69999, 65536, 1]], dtype=torch.int32, device=DEV)
    near = torch.tensor([[3, 0, 7]], dtype=torch.int32, device=DEV)
    k, v = bf16(rng, (600, H_kv, d)).to(DEV), bf16(rng, (600, H_kv, d)).to(DEV)
    q = bf16(rng, (3, 4, d)).to(DEV)
    res = []
    for cache, table in ((c, far), (small, near)):
        cache.write(k, v, offsets([600]), None, table)
        res.append(cache.attend(q, offsets([3]), i32([597]), table, d ** -0.5) +
                   cache.read(offsets([600]), None, table, 600))
    for a, b in zip(*res):
        assert torch.equal(a, b)


LONG_RUNS = [
    # sequences, longest context, new tokens, H, H_kv, d, page, window, sinks
    (120, 2500, 1, 16, 8, 128, 64, 0, 0),
    (120, 2500, 1, 16, 16, 64, 32, 0, 0),
    (90, 2500, 2, 16, 4, 128, 128, 0, 0),
    (90, 2500, 4, 8, 2, 64, 64, 700, 4),
    (40, 2500, 40, 8, 4, 128, 256, 0, 0),
    (30, 2500, 70, 8, 8, 64, 64, 300, 130),
]


@pytest.mark.parametrize("nseq,longest,new,H,H_kv,d,page,window,sinks", LONG_RUNS)
def test_many_tiles_a_cta(lib, nseq, longest, new, H, H_kv, d, page, window, sinks):
    """Batches that give every CTA a run of many key tiles and several items, against
    float64 attention (torch) of the values read back from the cache."""
    from precision_causal_attention_block_gb300 import flamia as fl
    from tests.serving_helpers import attend_tolerance, lse_tolerance, page_table, weight_error
    rng = np.random.default_rng(nseq + d + new)
    lens = [int(x) for x in np.exp(rng.uniform(np.log(new), np.log(longest), nseq))]
    n = [int(min(c, rng.integers(1, new + 1))) for c in lens]
    starts = [c - m for c, m in zip(lens, n)]
    t, pages = page_table(rng, lens, page)
    table = torch.from_numpy(t).to(DEV)
    cache = fl.KVCache(pages, page, H_kv, d)
    L, T = sum(lens), sum(n)
    g = torch.Generator(device=DEV).manual_seed(nseq)
    new_rows = lambda rows, h: torch.randn(rows, h, d, generator=g, device=DEV).to(torch.bfloat16)
    cache.write(new_rows(L, H_kv), new_rows(L, H_kv), offsets(lens), None, table)
    k, v = cache.read(offsets(lens), None, table, L)
    q = new_rows(T, H)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = cache.attend(q, offsets(n), i32(starts), table, d ** -0.5, window=window, sinks=sinks,
                          dev_status=st)
    assert int(st.item()) == 0
    weight = weight_error(T, nseq, H // H_kv)
    at = base = 0
    for b in range(nseq):
        qb = q[at:at + n[b]].double()
        kb, vb = k[base:base + lens[b]].double(), v[base:base + lens[b]].double()
        i = torch.arange(starts[b], lens[b], device=DEV)[:, None]
        j = torch.arange(lens[b], device=DEV)
        seen = j <= i
        if window:
            seen &= (j > i - window) | (j < sinks)
        x = torch.einsum("ihd,jhd->hij", qb, kb.repeat_interleave(H // H_kv, 1)) * d ** -0.5
        x = x.masked_fill(~seen, -torch.inf)
        p = torch.softmax(x, 2)
        vb = vb.repeat_interleave(H // H_kv, 1)
        ref, mass = torch.einsum("hij,jhd->ihd", p, vb), torch.einsum("hij,jhd->ihd", p, vb.abs())
        # a block's scale is at most 2 / 448 of its largest value
        top = 2 * p.amax(2).t()[..., None] * vb.abs().max()
        rl = torch.logsumexp(x, 2).cpu().numpy()
        qn, kn, rn, mass, top = (y.cpu().numpy() for y in (qb, kb, ref, mass, top))
        tol = attend_tolerance(qn, kn, d ** -0.5, lens[b], rn, weight, mass, top)
        err = np.abs(o[at:at + n[b]].double().cpu().numpy() - rn)
        assert (err <= tol).all(), (b, (err / tol).max())
        err = np.abs(lse[:, at:at + n[b]].double().cpu().numpy() - rl)
        assert (err <= lse_tolerance(qn, kn, d ** -0.5, rl)).all(), b
        at += n[b]
        base += lens[b]
