"""Calls of attend without a workspace that run at once: on two streams, from two
threads, captured and eager ones.  Nothing but the call's own workspace may be written."""
import threading

import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, bf16, i32, offsets

pytestmark = pytest.mark.gpu


def _setup(fl, seed, d=128, H=8, H_kv=4, ctx=9000):
    """A cache, and calls over it whose items are cut into many parts."""
    rng = np.random.default_rng(seed)
    pages = -(-ctx // 128)
    cache = fl.KVCache(pages, 128, H_kv, d)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
    x, y = (bf16(rng, (ctx, H_kv, d)).to(DEV) for _ in range(2))
    cache.write(x, y, offsets([ctx]), None, table)
    calls = []
    for n in (1, 3, 6, 150):  # 8, 8, 16 and 256 rows an item
        q = bf16(rng, (n, H, d)).to(DEV)
        args = (q, offsets([n]), i32([ctx - n]), table, d ** -0.5)
        calls.append((args, torch.empty_like(q), torch.empty(H, n, device=DEV)))
    return cache, calls


def _expected(cache, calls):
    out = []
    for args, _, _ in calls:
        o, lse = cache.attend(*args)
        torch.cuda.synchronize()
        out.append((o, lse))
    return out


def test_a_cache_holds_its_codes_and_scales_only(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    before = torch.cuda.memory_allocated()
    caches = [fl.KVCache(64, 64, 2, 128) for _ in range(8)]
    one = 2 * 64 * 2 * 64 * 129
    assert torch.cuda.memory_allocated() - before <= 8 * (one + 4 * 512)
    del caches


def test_streams_and_caches_at_once(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    cache, calls = _setup(fl, 1)
    want = _expected(cache, calls)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for rep in range(40):
        for s, (args, o, lse) in zip(streams, calls):
            with torch.cuda.stream(s):
                cache.attend(*args, o=o, lse=lse)
    torch.cuda.synchronize()
    for (_, o, lse), (wo, wl) in zip(calls, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_captured_calls_replayed_at_once(lib):
    """Graphs captured on one stream and replayed side by side, next to eager calls."""
    from precision_causal_attention_block_gb300 import flamia as fl
    cache, calls = _setup(fl, 2)
    want = _expected(cache, calls)
    graphs = []
    for args, o, lse in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                cache.attend(*args, o=o, lse=lse)
        graphs.append(g)
    for _, o, lse in calls:
        o.zero_()
        lse.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    eager = []
    for rep in range(15):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager.append(cache.attend(*calls[rep % 4][0]))
    torch.cuda.synchronize()
    for (_, o, lse), (wo, wl) in zip(calls, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)
    for rep, (o, lse) in enumerate(eager):
        assert torch.equal(o, want[rep % 4][0]) and torch.equal(lse, want[rep % 4][1])


def test_threads_on_one_stream(lib):
    """The library is called without the interpreter's lock, so the two kernels of a
    call may have another thread's between them."""
    from precision_causal_attention_block_gb300 import flamia as fl
    cache, calls = _setup(fl, 3)
    want = _expected(cache, calls)
    torch.cuda.synchronize()
    errors = []

    def work(args, o, lse):
        try:
            for _ in range(200):
                cache.attend(*args, o=o, lse=lse)
        except Exception as e:  # (seen by the assertion below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for (_, o, lse), (wo, wl) in zip(calls, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_a_streams_workspace_stays(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    cache, calls = _setup(fl, 4)
    other, _ = _setup(fl, 5, d=64)
    at = cache._ws.data_ptr()
    for args, _, _ in calls:
        cache.attend(*args)
        assert cache._ws.data_ptr() == other._ws.data_ptr() == at
    with torch.cuda.stream(torch.cuda.Stream()):
        assert cache._ws.data_ptr() != at
