"""The entry points of rotary axes, pages and shared prefixes refuse bad arguments on the
host: no kernel is launched (there need not be a GPU)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    from precision_causal_attention_block_gb300 import build, flamia
    build.build()
    lib = flamia.load()
    buf = np.zeros(1 << 16, dtype=np.uint8)
    at = (buf.ctypes.data + 255) // 256 * 256
    before = lib.flamia_debug_launch_count()
    yield flamia, lib, at, buf
    assert lib.flamia_debug_launch_count() == before


def _call(fn, a, kw):
    assert not set(kw) - set(a)
    return fn(*{**a, **kw}.values())


def _cache(fl, at, **kw):
    a = dict(k_codes=at, k_scales=at, v_codes=at, v_scales=at, num_pages=4, page_size=64, H_kv=2, d=64)
    a.update(kw)
    return fl.KVCacheStruct(*a.values())


def test_rope_axes(env):
    _, lib, at, _ = env
    a = dict(q_in=at, q_out=at, qis=256, qos=256, k_in=at, k_out=at, kis=128, kos=128, T=2, H=4, H_kv=2, d=64, turns=at,
             axes=at, rot=64, m=1.0, flags=0, positions=at, pos_stride=2, naxes=3, cu=at, n=1, st=None, s=None)
    run = lambda **kw: _call(lib.flamia_rope_axes, a, kw)
    assert run(T=0) == OK
    for kw in (dict(d=96), dict(rot=24), dict(rot=128), dict(flags=1), dict(flags=0x8000)):
        assert run(**kw) == UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(n=0), dict(H=0), dict(H_kv=-1), dict(q_in=None), dict(turns=None),
               dict(axes=None), dict(positions=None), dict(positions=at + 2), dict(naxes=0), dict(naxes=33),
               dict(pos_stride=-1), dict(pos_stride=1 << 40), dict(cu=None), dict(qis=260), dict(qos=248),
               dict(qis=264), dict(m=float("inf"))):
        assert run(**kw) == INVALID, kw


def test_pages_copy(env):
    fl, lib, at, _ = env
    c = lambda **kw: ctypes.byref(_cache(fl, at, **kw))
    run = lambda **kw: _call(lib.flamia_pages_copy, dict(f=c(), t=c(), src=at, dst=at, n=3, st=None, s=None), kw)
    assert run(n=0) == OK
    for kw in (dict(f=None), dict(t=None), dict(t=c(page_size=32)), dict(t=c(H_kv=4)), dict(t=c(d=128)), dict(n=-1),
               dict(src=None), dict(dst=None), dict(dst=at + 1), dict(f=c(k_codes=at + 16))):
        assert run(**kw) == INVALID, kw
    assert run(f=c(d=96), t=c(d=96)) == UNSUPPORTED
    assert run(f=c(page_size=48), t=c(page_size=48)) == UNSUPPORTED


def test_pages_fork(env):
    _, lib, at, _ = env
    need = lib.flamia_pages_fork_workspace_bytes(3, 8)
    assert need >= 3 * 8 * 4
    a = dict(refs=at, pages=4, table=at, stride=8, nseq=4, page=64, parents=at, children=at, n=3, lens=at, ws=at,
             size=need, st=None, s=None)
    run = lambda **kw: _call(lib.flamia_pages_fork, a, kw)
    assert run(n=0) == OK and run(n=0, children=None, ws=None) == OK
    for kw in (dict(refs=None), dict(pages=0), dict(table=None), dict(stride=0), dict(nseq=0), dict(nseq=65537),
               dict(page=0), dict(children=None), dict(children=at + 2), dict(parents=at + 1), dict(n=-1), dict(n=5),
               dict(lens=None), dict(ws=None), dict(ws=at + 128), dict(nseq=65536, stride=1 << 15)):
        assert run(**kw) == INVALID, kw
    assert run(size=need - 1) == WORKSPACE
    for args in ((0, 8), (3, 0), (-1, 8), (65537, 1)):
        assert lib.flamia_pages_fork_workspace_bytes(*args) == 0


def test_pages_reserve(env):
    fl, lib, at, _ = env
    need = lib.flamia_pages_reserve_workspace_bytes(10, 4, 8, 64)
    assert need > 0
    c = lambda **kw: ctypes.byref(_cache(fl, at, **kw))
    a = dict(c=c(), refs=at, table=at, stride=8, nseq=4, T=10, cu=at, starts=None, granted=None, ws=at, size=need, st=None, s=None)
    run = lambda **kw: _call(lib.flamia_pages_reserve, a, kw)
    assert run(T=0) == OK and run(T=0, cu=None, ws=None) == OK
    for kw in (dict(c=None), dict(refs=None), dict(refs=at + 1), dict(table=None), dict(stride=0), dict(nseq=0),
               dict(nseq=65537), dict(T=-1), dict(T=(1 << 20) + 1), dict(cu=None), dict(ws=None), dict(ws=at + 4),
               dict(c=c(num_pages=0)), dict(granted=at), dict(granted=at + 2)):
        assert run(**kw) == INVALID, kw
    assert run(size=need - 1) == WORKSPACE and run(c=c(d=32)) == UNSUPPORTED
    for args in ((-1, 4, 8, 64), (10, 0, 8, 64), (10, 4, 0, 64), (10, 4, 8, 0), (1 << 21, 4, 8, 64)):
        assert lib.flamia_pages_reserve_workspace_bytes(*args) == 0
    # a token a sequence: a slot each, and as many rows of a copy list
    assert lib.flamia_pages_reserve_workspace_bytes(1000, 1000, 2048, 64) < 1 << 20


def test_pages_compact(env):
    fl, lib, at, _ = env
    need = lib.flamia_pages_compact_workspace_bytes(4)
    c = lambda **kw: ctypes.byref(_cache(fl, at, **kw))
    a = dict(c=c(), refs=at, table=at, stride=8, nseq=4, live=None, ws=at, size=need, st=None, s=None)
    run = lambda **kw: _call(lib.flamia_pages_compact, a, kw)
    for kw in (dict(c=None), dict(refs=None), dict(table=None), dict(stride=0), dict(nseq=0), dict(live=at + 2),
               dict(ws=None), dict(ws=at + 8)):
        assert run(**kw) == INVALID, kw
    assert run(size=need - 1) == WORKSPACE
    assert lib.flamia_pages_compact_workspace_bytes(0) == 0


def test_attend_prefix(env):
    fl, lib, at, _ = env
    c = lambda **kw: ctypes.byref(_cache(fl, at, **kw))
    size = lambda *x: lib.flamia_attn_cache_prefix_workspace_bytes(*x)
    always = fl.FLAG_PREFIX_ALWAYS
    need = size(4, 3, 4, 2, 64, 300, always)
    a = dict(c=c(), q=at, qs=256, T=4, H=4, cu=at, n=3, starts=None, table=at, stride=8, prefix=300, scale=0.125,
             flags=always, o=at, lse=None, ws=at, size=need, st=None, s=None)
    run = lambda **kw: _call(lib.flamia_attn_cache_prefix, a, kw)
    assert run(T=0) == OK
    for kw in (dict(c=None), dict(q=None), dict(q=at + 2), dict(qs=260), dict(T=-1), dict(H=0), dict(H=5), dict(cu=None),
               dict(n=0), dict(table=None), dict(stride=0), dict(prefix=-1), dict(scale=0.0), dict(scale=float("nan")),
               dict(o=None), dict(o=at + 8), dict(lse=at + 2), dict(ws=None), dict(ws=at + 16)):
        assert run(**kw) == INVALID, kw
    for kw in (dict(flags=1), dict(flags=0x4000), dict(c=c(d=32))):
        assert run(**kw) == UNSUPPORTED, kw
    assert run(size=need - 1) == WORKSPACE
    # calls that gain nothing take the plain call's workspace
    plain = lib.flamia_attn_cache_workspace_bytes
    assert size(4, 3, 4, 2, 64, 300, 0) == plain(4, 3, 4, 2, 64)
    assert size(4, 1, 4, 2, 64, 1 << 20, always) == plain(4, 1, 4, 2, 64)
    assert size(4, 3, 4, 2, 64, 127, always) == plain(4, 3, 4, 2, 64)
    assert size(400, 2, 4, 2, 64, 300, always) == plain(400, 2, 4, 2, 64)
    assert size(96, 96, 32, 8, 128, 16421, 0) != plain(96, 96, 32, 8, 128)
    for x in ((4, 3, 4, 2, 96, 300, 0), (4, 3, 4, 3, 64, 300, 0), (4, 3, 4, 2, 64, -1, 0), (4, 3, 4, 2, 64, 300, 2)):
        assert size(*x) == 0


def test_axes_of_pairs():
    from precision_causal_attention_block_gb300 import flamia as fl
    assert fl.rope_axes([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert fl.rope_axes([2, 1, 3], cyclic=True) == [0, 1, 2, 0, 2, 2]
    assert fl.rope_axes([0, 2], cyclic=True) == fl.rope_axes([0, 2]) == [1, 1]
    for bad in ([], [-1, 2]):
        with pytest.raises(ValueError):
            fl.rope_axes(bad)
    w = fl.rope_frequencies(16)
    assert fl.Rotary(w, device="cpu", axes=[0, 0, 1, 1, 2, 2, 2, 2]).naxes == 3
    for bad in ([0] * 7, [0] * 7 + [-1], [0] * 7 + [8], []):
        with pytest.raises(ValueError):
            fl.Rotary(w, device="cpu", axes=bad)
    q, cu = torch.zeros(2, 1, 16, dtype=torch.bfloat16), torch.tensor([0, 2], dtype=torch.int32)
    pos = torch.zeros(1, 2, dtype=torch.int32)
    for rope, kw in ((fl.Rotary(w, device="cpu"), dict(positions=pos)), (fl.Rotary(w, device="cpu", axes=[0] * 8), {}),
                     (fl.Rotary(w, device="cpu", axes=[0] * 8), dict(positions=pos, starts=cu[:1]))):
        with pytest.raises(RuntimeError, match="positions"):
            rope(q, None, cu, **kw)


def test_calls_and_pools_that_do_not_fit():
    """What the Python objects refuse before any call."""
    import types
    from precision_causal_attention_block_gb300 import flamia as fl
    cache = types.SimpleNamespace(num_pages=4, k_codes=torch.zeros(1), device_index=-1)
    table, refs = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    pool = fl.PagePool.from_buffers(cache, table, refs)
    for t, r in ((table.long(), refs), (table[:, :2], refs), (table[0], refs), (table, refs[:3]), (table, refs.float())):
        with pytest.raises(RuntimeError):
            fl.PagePool.from_buffers(cache, t, r)
    for kw in (dict(nseq=3), dict(nseq=2, other=True)):
        other = types.SimpleNamespace(**vars(cache)) if kw.pop("other", False) else cache
        with pytest.raises(RuntimeError, match="pool"):
            fl.DecodeCall(other, 1, H=1, softmax_scale=1.0, pool=pool, **kw)


def test_the_binding_s_page_calls(monkeypatch):
    """Counts that do not match are refused before the library is called."""
    import types
    from precision_causal_attention_block_gb300 import flamia as fl
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or (64 if name.endswith("bytes") else 0)

    monkeypatch.setattr(fl, "_LIB", Lib())
    monkeypatch.setattr(fl, "_current", lambda: (-1, 0))
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    cache = types.SimpleNamespace(num_pages=4, page_size=32, k_codes=torch.zeros(1), device_index=-1, _ref=None)
    pool = fl.PagePool.from_buffers(cache, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    pool.fork(i(2), i(2), i(2))
    assert [c[0] for c in calls] == ["flamia_pages_fork_workspace_bytes", "flamia_pages_fork"]
    pool.fork(None, i(2), i(2))
    pool.reserve(i(3), i(2), 5)
    assert calls[-1][0] == "flamia_pages_reserve" and calls[-1][1][5] == 5
    n = len(calls)
    pool.fork(i(0), i(0), i(2))  # nothing to do
    for bad in (lambda: pool.fork(i(3), i(2), i(2)), lambda: pool.fork(i(0), i(2), i(2)), lambda: pool.fork(i(2), i(2), i(3)),
                lambda: pool.fork(i(2).long(), i(2), i(2)), lambda: pool.reserve(i(2), i(2)), lambda: pool.reserve(i(3), i(3)),
                lambda: pool.reserve(i(3), i(2), 5, i(2)),
                lambda: pool.compact(i(2)), lambda: fl.flamia_pages_copy(cache, cache, i(2), i(3)),
                lambda: fl.flamia_pages_copy(cache, cache, i(0), i(3))):
        with pytest.raises(RuntimeError):
            bad()
    assert len(calls) == n


CSRC = os.path.join(ROOT, "precision_causal_attention_block_gb300", "csrc")
FILES = ["pages.cu", "attn_prefix.cu", "attn_prefix_rows.cu", "attend_rows.cuh"]


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_sources_read_no_input_before_the_wait():
    """As for the other serving kernels: no read-only loads, and every kernel waits for the
    one before it in the stream."""
    for name in FILES:
        code = _code(name)
        assert not re.search(r"__ldg\b|\.nc\b|__restrict__|__restrict\b", code), name
        for m in re.finditer(r"__global__ void __launch_bounds__", code):
            body = code[m.start():]
            end = body.find("__global__ void", 1)
            assert "wait_for_previous();" in (body[:end] if end > 0 else body), (name, body[:120])


def test_products_in_flight_end_before_their_memory_goes():
    code = _code("attn_prefix_rows.cu")
    failed = [code[m.end():m.end() + 400] for m in re.finditer(r"if \(!ok\) \{", code)]
    assert any(re.search(r"tc_commit_w\(smem_u32\(&sm\.drained\[w\]\)\);.*mbar_wait_w\(smem_u32\(&sm\.drained\[w\]\), 0\);",
                         f, re.S) for f in failed)
