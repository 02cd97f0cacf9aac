"""Offsets that are not those of packed sequences: reserve takes no page, copies nothing and
grants nothing, so that a step over a pool cannot write into pages that others hold."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, bf16, i32, offsets

pytestmark = pytest.mark.gpu

# copies by the CTA that keeps the books, or by a kernel behind it
FORMS = [(32, 1, 64), (256, 4, 128)]


def _arrays(cache):
    return [cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales]


def _forked(fl, page, H_kv, d):
    """Sequence 1 holds seven pages, sequence 2 shares them, sequence 0 is empty."""
    rng = np.random.default_rng(page)
    cache = fl.KVCache(24, page, H_kv, d)
    pool = fl.PagePool(cache, 3, 8)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    n = [0, 7 * page, 0]
    x, y = (bf16(rng, (7 * page, H_kv, d)).to(DEV) for _ in range(2))
    pool.reserve(offsets(n), lens)
    cache.write(x, y, offsets(n), lens, pool.page_table)
    lens[1] = 7 * page
    pool.fork(i32([1]), i32([2]), lens)
    pool.check_status()
    return rng, cache, pool, lens


@pytest.mark.parametrize("page,H_kv,d", FORMS)
def test_a_step_with_overlapping_ranges_leaves_shared_pages(lib, page, H_kv, d):
    """Two sequences claim the same tokens, more slots than a call of so many tokens can
    touch; the second one's last blocks lie in pages that its parent holds."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng, cache, pool, lens = _forked(fl, page, H_kv, d)
    T, H = 6 * page + page // 4, 2 * H_kv
    call = fl.DecodeCall(cache, T, 3, H, d ** -0.5, pool=pool)
    call.o.fill_(7)
    pages = pool.page_table[1, :7].long()
    held = [x[pages].clone() for x in _arrays(cache)]
    books = pool.page_table.clone(), pool.refs.clone()
    q, k, v = (bf16(rng, (T, h, d), 50.0).to(DEV) for h in (H, H_kv, H_kv))
    call(q, k, v, i32([0, T, 0, T]), i32([0, 0, 0]))
    with pytest.raises(RuntimeError, match="0x1$"):
        call.check_status()
    assert all(torch.equal(x[pages], y) for x, y in zip(_arrays(cache), held))
    assert (call.granted == 0).all() and (call.o == 7).all()
    assert torch.equal(pool.page_table, books[0]) and torch.equal(pool.refs, books[1])


@pytest.mark.parametrize("page,H_kv,d", FORMS)
@pytest.mark.parametrize("cu", [[0, 90, 40, 100], [3, 10, 20, 30], [0, 10, 20, 300], [0, -5, 10, 20],
                                [-1, 10, 20, 30], [0, 10, 20, 19], [0, 1 << 30, 1 << 30, -(1 << 30)]])
def test_reserve_takes_nothing(lib, page, H_kv, d, cu):
    from precision_causal_attention_block_gb300 import flamia as fl
    _, cache, pool, lens = _forked(fl, page, H_kv, d)
    before = [x.clone() for x in _arrays(cache)]
    books = pool.page_table.clone(), pool.refs.clone()
    granted = i32([9] * 4)
    pool.reserve(i32(cu), i32([0, page, 5]), T=200, granted=granted)
    assert int(pool.status.item()) == fl.DEV_BAD_SEQLENS
    assert (granted == 0).all()
    assert torch.equal(pool.page_table, books[0]) and torch.equal(pool.refs, books[1])
    assert all(map(torch.equal, _arrays(cache), before))
    # the pool goes on from there
    pool.status.zero_()
    pool.reserve(offsets([1, 0, 1]), lens, T=200, granted=granted)
    pool.check_status()
    assert granted.tolist() == [0, 1, 1, 2] and (pool.refs > 0).sum() == 9
