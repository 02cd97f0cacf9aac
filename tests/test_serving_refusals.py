"""The rotary and cache entry points refuse bad arguments on the host: no
kernel is launched (there need not be a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


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


def _rope(lib, at, **kw):
    a = dict(q_in=at, q_out=at, qis=256, qos=256, k_in=at, k_out=at, kis=128, kos=128, T=2, H=4,
             H_kv=2, d=64, turns=at, rot=64, m=1.0, flags=0, cu=at, n=1, starts=None, st=None,
             s=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.flamia_rope(*a.values())


def test_rope(env):
    _, lib, at, _ = env
    assert _rope(lib, at, T=0) == OK
    for kw in (dict(d=96), dict(rot=24), dict(rot=0), dict(rot=128), dict(flags=1),
               dict(flags=0x8000)):
        assert _rope(lib, at, **kw) == UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(n=0), dict(n=(1 << 20) + 1), dict(H=0),
               dict(H=4097), dict(H_kv=-1), dict(q_in=None), dict(q_out=None), dict(k_in=None),
               dict(k_out=None), dict(turns=None), dict(cu=None), dict(q_in=at + 8),
               dict(k_out=at + 2), dict(turns=at + 4), dict(qis=260), dict(qos=248), dict(kos=64),
               dict(qis=264), dict(kis=-128), dict(m=float("nan"))):
        assert _rope(lib, at, **kw) == INVALID, kw


def _cache(fl, at, **kw):
    a = dict(k_codes=at, k_scales=at, v_codes=at, v_scales=at, num_pages=4, page_size=64, H_kv=2,
             d=64)
    a.update(kw)
    return fl.KVCacheStruct(*a.values())


def _write(fl, lib, at, cache=None, read=False, **kw):
    a = dict(k=at, ks=128, v=at, vs=128, T=2, cu=at, n=1, starts=None, table=at, stride=1)
    if not read:
        a["format"] = 0
    a.update(st=None, s=None)
    assert not set(kw) - set(a)
    a.update(kw)
    c = _cache(fl, at, **(cache or {}))
    fn = lib.flamia_cache_read if read else lib.flamia_cache_write
    return fn(ctypes.byref(c), *a.values())


BAD_CACHE = [(dict(d=80), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED),
             (dict(page_size=48), UNSUPPORTED), (dict(page_size=192 + 32), UNSUPPORTED),
             (dict(page_size=(1 << 20) + 128), UNSUPPORTED), (dict(num_pages=0), INVALID),
             (dict(H_kv=0), INVALID), (dict(H_kv=4097), INVALID),
             (dict(num_pages=1 << 30, H_kv=2), INVALID), (dict(k_codes=None), INVALID),
             (dict(v_scales=None), INVALID)]


@pytest.mark.parametrize("read", [False, True])
def test_cache_write_and_read(env, read):
    fl, lib, at, _ = env
    assert _write(fl, lib, at, read=read, T=0) == OK
    for c, want in BAD_CACHE + [(dict(v_codes=at + 64), INVALID), (dict(k_scales=at + 16), INVALID)]:
        assert _write(fl, lib, at, cache=c, read=read) == want, c
    for kw in (dict(T=-1), dict(n=0), dict(stride=0), dict(k=None), dict(v=None), dict(cu=None),
               dict(table=None), dict(k=at + 8), dict(vs=132), dict(ks=-128)):
        assert _write(fl, lib, at, read=read, **kw) == INVALID, kw
    if read:
        assert _write(fl, lib, at, read=True, ks=64) == INVALID
    else:
        for f in (1, 0x10, 0x30, 2):
            assert _write(fl, lib, at, format=f) == UNSUPPORTED


def _attend(fl, lib, at, cache=None, null_cache=False, **kw):
    a = dict(q=at, qs=256, T=2, H=4, cu=at, n=1, starts=None, table=at, stride=1, scale=0.125,
             window=0, sinks=0, o=at, lse=at, ws=at, ws_bytes=1 << 40, st=None, s=None)
    assert not set(kw) - set(a)
    a.update(kw)
    c = _cache(fl, at, **(cache or {}))
    return lib.flamia_attn_cache(None if null_cache else ctypes.byref(c), *a.values())


def test_attend(env):
    fl, lib, at, _ = env
    assert _attend(fl, lib, at, T=0) == OK
    assert _attend(fl, lib, at, null_cache=True) == INVALID
    for c, want in BAD_CACHE:
        assert _attend(fl, lib, at, cache=c) == want, c
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(n=0), dict(H=3), dict(H=0), dict(H=4098),
               dict(stride=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(sinks=4),
               dict(q=None), dict(q=at + 8), dict(qs=12), dict(cu=None), dict(table=None),
               dict(o=None), dict(o=at + 8), dict(ws=None), dict(ws=at + 128), dict(lse=at + 2)):
        assert _attend(fl, lib, at, **kw) == INVALID, kw
    assert _attend(fl, lib, at, ws_bytes=0) == WORKSPACE
    size = fl.flamia_attn_cache_workspace_bytes
    assert size(64, 64, 32, 8, 128) > 0 and size(0, 1, 32, 8, 128) > 0
    for args in ((64, 64, 32, 8, 96), (64, 0, 32, 8, 128), (64, 64, 30, 8, 128),
                 (-1, 64, 32, 8, 128), (64, 64, 0, 8, 128), (64, 64, 32, 0, 128)):
        assert size(*args) == 0, args


def test_python_binding_refuses_before_the_library(env):
    fl = env[0]
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    rot = fl.Rotary(fl.rope_frequencies(64), device="cpu")
    with pytest.raises(RuntimeError, match="CUDA"):
        rot(x, x, cu)
    with pytest.raises(RuntimeError, match="BF16"):
        rot(x.float(), None, cu)
    with pytest.raises(RuntimeError, match="contiguous"):
        rot(x.transpose(1, 2), None, cu)
    with pytest.raises(RuntimeError, match="CUDA"):
        fl.KVCache(2, 64, 4, 64, device="cpu")
    with pytest.raises(RuntimeError, match="pages"):
        fl.KVCache.from_buffers(x, x, x, x)
    with pytest.raises(ValueError):
        fl.Rotary([1.0, float("inf")], device="cpu")
