"""Captured calls on pools whose copies and rows are too many for the CTA that keeps the books:
a second kernel behind it copies pages or writes rows, and takes what it does from memory of the
graph's own."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, bf16, i32, offsets
from tests.test_gpu_pages import Both

pytestmark = pytest.mark.gpu


def _captured(f):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = f()
    torch.cuda.current_stream().wait_stream(side)
    return g, out


@pytest.mark.parametrize("pages,page,H_kv,d,nseq,width", [(60, 256, 4, 128, 5, 1400),  # all of them
                                                          (60, 256, 4, 128, 5, 8),     # copies
                                                          (60, 32, 1, 64, 5, 7000)])   # rows
def test_books_with_a_kernel_behind(lib, pages, page, H_kv, d, nseq, width):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(width)
    both = Both(fl, rng, pages, page, H_kv, d, nseq, width)
    both.append(rng, [40, page + 38, 0, 0, 0])
    parents, children = i32([0, 1, 0]), i32([2, 3, 4])
    cu, lens, granted = offsets([0, 0, 1, 1, 1]), both.lens, i32([5] * (nseq + 1))

    def step():
        both.pool.fork(parents, children, lens)
        both.pool.reserve(cu, lens, granted=granted)
        return both.pool.compact()

    g, live = _captured(step)
    both.check()  # (nothing has run)
    # (the second graph's workspaces are others: it runs between the first one's replays)
    g2, live2 = _captured(step)
    for i, (p, c) in enumerate((([0, 1, 0], [2, 3, 4]), ([1, -1, 0], [2, 3, 0]), ([2, 2, 1], [3, 4, 2]),
                                ([4, 0, 1], [1, 2, 3]))):
        parents.copy_(i32(p))
        children.copy_(i32(c))
        (g2 if i & 1 else g).replay()
        both.ref.fork(p, c, both.n)
        assert both.ref.reserve([0, 0, 1, 1, 1], both.n)
        assert int((live2 if i & 1 else live).item()) == both.ref.compact()
        assert torch.equal(granted, cu)
        both.check()
    both.pool.check_status()


@pytest.mark.parametrize("always", [False, True])
def test_decode_steps_copy_pages_behind_the_books(lib, always):
    """A step over forked sequences of large pages, captured and replayed across a page's end:
    the same bits as eager steps."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(1)
    H, H_kv, d, page, prompt, nseq = 8, 4, 128, 256, 1000, 6

    def build():
        cache = fl.KVCache(40, page, H_kv, d)
        pool = fl.PagePool(cache, nseq, 6)
        lens = torch.zeros(nseq, dtype=torch.int32, device=DEV)
        x = bf16(np.random.default_rng(2), (prompt, H_kv, d)).to(DEV)
        cu = offsets([prompt] + [0] * (nseq - 1))
        pool.reserve(cu, lens)
        cache.write(x, x, cu, lens, pool.page_table)
        lens[0] = prompt
        pool.fork(i32([0] * (nseq - 1)), i32(range(1, nseq)), lens)
        return cache, pool, lens, fl.DecodeCall(cache, nseq, nseq, H, d ** -0.5, pool=pool, prefix=prompt,
                                                rope=fl.Rotary(fl.rope_frequencies(d)), always_share=always)

    cu = offsets([1] * nseq)
    q, k, v = (torch.zeros(nseq, h, d, dtype=torch.bfloat16, device=DEV) for h in (H, H_kv, H_kv))
    c1, p1, l1, s1 = build()
    c2, p2, l2, s2 = build()

    def step():
        s1(q, k, v, cu, l1)
        l1.add_(s1.granted.diff())

    g, _ = _captured(step)
    for _ in range(30):
        for t, h in ((q, H), (k, H_kv), (v, H_kv)):
            t.copy_(bf16(rng, (nseq, h, d)))
        g.replay()
        s2(q, k, v, cu, l2)
        l2.add_(s2.granted.diff())
        assert torch.equal(s1.o, s2.o) and torch.equal(s1.lse, s2.lse)
    s1.check_status()
    s2.check_status()
    assert l1.tolist() == l2.tolist() == [prompt + 30] * nseq
    assert torch.equal(p1.page_table, p2.page_table) and torch.equal(p1.refs, p2.refs)
    assert torch.equal(c1.k_codes, c2.k_codes) and torch.equal(c1.v_scales, c2.v_scales)
