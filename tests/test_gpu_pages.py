"""Pages of the cache against the oracle's books, bit for bit: page table, counts,
lengths and every byte of the pool."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.serving_helpers import DEV, i32, offsets

pytestmark = pytest.mark.gpu


def _arrays(cache):
    return [cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales]


def _filled(fl, rng, pages, page, H_kv, d):
    cache = fl.KVCache(pages, page, H_kv, d)
    for x in _arrays(cache):
        x.copy_(torch.from_numpy(rng.integers(0, 256, x.shape, dtype=np.uint8)))
    return cache


class Both:
    """A pool on the GPU and the oracle's."""

    def __init__(self, fl, rng, pages, page, H_kv, d, nseq, width):
        self.cache = _filled(fl, rng, pages, page, H_kv, d)
        self.pool = fl.PagePool(self.cache, nseq, width)
        self.lens = torch.zeros(nseq, dtype=torch.int32, device=DEV)
        self.n = np.zeros(nseq, dtype=np.int64)
        self.ref = S.Pages(page, np.full((nseq, width), -1), np.zeros(pages, dtype=int),
                           [x.cpu().numpy().copy() for x in _arrays(self.cache)])

    def check(self):
        assert np.array_equal(self.pool.page_table.cpu().numpy(), self.ref.table)
        assert np.array_equal(self.pool.refs.cpu().numpy(), self.ref.refs)
        assert np.array_equal(self.lens.cpu().numpy(), self.n)
        for x, y in zip(_arrays(self.cache), self.ref.arrays):
            assert np.array_equal(x.cpu().numpy(), y)
        # the counts are those of the table
        t = self.ref.table
        assert np.array_equal(np.bincount(t[t >= 0], minlength=len(self.ref.refs)), self.ref.refs)

    def fork(self, parents, children):
        self.pool.fork(None if parents is None else i32(parents), i32(children), self.lens)
        self.ref.fork([-1] * len(children) if parents is None else parents, children, self.n)

    def append(self, rng, n):
        """n[b] new tokens a sequence: pages, then random rows in them."""
        self.pool.reserve(offsets(n), self.lens)
        ok = self.ref.reserve(n, self.n)
        if not ok:
            return False
        for b, c in enumerate(n):
            for p in range(self.n[b], self.n[b] + c):
                at = self.ref.table[b, p // self.ref.page]
                for x, y in zip(_arrays(self.cache), self.ref.arrays):
                    row = rng.integers(0, 256, y[at, :, p % self.ref.page].shape, dtype=np.uint8)
                    y[at, :, p % self.ref.page] = row
                    x[int(at), :, p % self.ref.page] = torch.from_numpy(row).to(DEV)
        self.n += np.asarray(n)
        self.lens += i32(n)
        return True


@pytest.mark.parametrize("pages,page,H_kv,d,n", [(9, 32, 1, 64, 4), (40, 64, 3, 128, 17),
                                                 (7, 256, 2, 64, 3), (300, 32, 5, 128, 150),
                                                 (5, 640, 1, 128, 2)])
def test_copy(lib, pages, page, H_kv, d, n):
    """Within a cache and to another one; pairs with a negative entry are left out and
    pages outside the pool reported."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(pages)
    a, b = _filled(fl, rng, pages, page, H_kv, d), _filled(fl, rng, pages + 3, page, H_kv, d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for source, target in ((a, a), (a, b), (b, a)):
        order = rng.permutation(pages)
        src, dst = order[:n].copy(), order[n:2 * n].copy()
        src[0] = -1
        dst[1] = -5
        ref = S.Pages(page, [[-1]], [0], [x.cpu().numpy().copy() for x in _arrays(target)])
        if source is target:
            ref.copy(src, dst)
        else:
            for i, j in zip(src, dst):
                if i >= 0 and j >= 0:
                    for x, y in zip(ref.arrays, _arrays(source)):
                        x[j] = y[int(i)].cpu().numpy()
        target.copy_pages(i32(src), i32(dst), source=None if source is target else source,
                          dev_status=status)
        for x, y in zip(_arrays(target), ref.arrays):
            assert np.array_equal(x.cpu().numpy(), y)
        assert status.item() == 0
    before = [x.clone() for x in _arrays(a)]
    a.copy_pages(i32([0, pages, 1 << 30]), i32([pages, 1, 2]), dev_status=status)
    assert status.item() == fl.DEV_BAD_PAGE
    a.copy_pages(i32([]), i32([]))
    assert all(torch.equal(x, y) for x, y in zip(before, _arrays(a)))


@pytest.mark.parametrize("page,H_kv,d,seed", [(32, 2, 64, 0), (64, 1, 128, 1), (256, 3, 64, 2),
                                                 (128, 2, 128, 3), (256, 2, 128, 4)])
def test_long_stories(lib, page, H_kv, d, seed):
    """Forks, new orders, truncations, ends and compactions in random turns."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(seed)
    nseq, width = 7, 6
    both = Both(fl, rng, 44, page, H_kv, d, nseq, width)
    assert both.append(rng, [3 * page - 5, 0, page, 1, 0, 0, 0])
    both.check()
    for _ in range(40):
        what = rng.integers(0, 5)
        if what == 0:
            k = int(rng.integers(1, nseq + 1))
            both.fork([int(x) for x in rng.integers(-1, nseq, k)],
                      [int(x) for x in rng.permutation(nseq)[:k]])
        elif what == 1:  # a new order of all
            both.fork([int(x) for x in rng.integers(0, nseq, nseq)], list(range(nseq)))
        elif what == 2:
            both.fork(None, [int(rng.integers(0, nseq))])
        elif what == 3:
            live = both.pool.compact()
            assert int(live.item()) == both.ref.compact()
        else:
            cut = rng.random(nseq) < 0.2  # drafted tokens that were not taken
            both.n = np.where(cut, both.n // 2, both.n)
            both.lens.copy_(i32(both.n))
            room = width * page - both.n
            n = [int(min(r, rng.choice([0, 0, 1, 1, page // 2, page + 3]))) for r in room]
            both.append(rng, n)
        both.check()
    assert int(both.pool.status.item()) & ~fl.DEV_CAPACITY == 0


def test_the_last_user_keeps_a_page(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(5)
    both = Both(fl, rng, 20, 32, 2, 64, 6, 3)
    both.append(rng, [40, 0, 0, 0, 0, 0])
    both.fork([0, 0, 0, 0], [1, 2, 3, 4])
    both.check()
    shared = int(both.ref.table[0, 1])
    assert both.ref.refs[shared] == 5
    both.append(rng, [1, 0, 1, 1, 0, 0])  # 1 and 4 still hold it: three copies
    both.check()
    assert both.ref.refs[shared] == 2
    both.append(rng, [0, 1, 0, 0, 1, 0])  # both here: one copy, the last keeps it
    both.check()
    assert both.ref.table[4, 1] == shared and both.ref.refs[shared] == 1
    assert both.ref.refs[both.ref.table[0, 0]] == 5
    both.pool.check_status()


@pytest.mark.parametrize("nseq,width", [(129, 4), (40, 130), (128, 32), (127, 33)])
def test_forks_of_many_slots(lib, nseq, width):
    """One CTA keeps the rows, or a launch reads and a launch writes them: an order of all
    sequences, some of them ended and some twice parents."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(nseq)
    both = Both(fl, rng, nseq * 3 + width, 32, 1, 64, nseq, width)
    n = rng.integers(0, 65, nseq)
    n[3] = 32 * width
    both.append(np.random.default_rng(1), [int(min(x, 40)) if i != 3 else 32 for i, x in enumerate(n)])
    for _ in range(3):
        both.fork([int(x) for x in rng.integers(-1, nseq, nseq)], [int(x) for x in rng.permutation(nseq)])
        both.check()
        k = nseq // 2
        both.fork([int(x) for x in rng.integers(0, nseq, k)], [int(x) for x in rng.integers(-1, nseq, k)])
        both.check()
    both.pool.check_status()


def test_no_free_page_changes_nothing(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(6)
    both = Both(fl, rng, 5, 32, 1, 64, 4, 4)
    assert both.append(rng, [40, 0, 33, 0])  # four pages
    both.fork([0], [1])
    both.check()
    # a copy for one of 0 and 1 (together they leave the shared page), a page for 3 x 2
    assert not both.append(rng, [1, 1, 0, 64])
    assert int(both.pool.status.item()) == fl.DEV_CAPACITY
    both.check()
    with pytest.raises(RuntimeError, match="0x2"):
        both.pool.check_status()
    both.pool.status.zero_()
    assert both.append(rng, [1, 1, 0, 0])  # the fifth page
    both.check()
    both.pool.check_status()
    assert (both.pool.refs > 0).all()


def test_many_sequences_and_long_prompts(lib):
    """More sequences than the planning CTA has threads, slots in the thousands, and a
    pool of more pages than it looks at in a round."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(7)
    nseq, page, pages = 2500, 32, 20011
    both = Both(fl, rng, pages, page, 1, 64, nseq, 300)
    held = rng.permutation(pages)[:9000]  # pages that are nobody's here
    both.ref.refs[held] = 1
    both.pool.refs[torch.from_numpy(held).to(DEV)] = 1
    n = rng.integers(0, 60, nseq)
    n[17], n[2400] = 9000, 7777
    both.pool.reserve(offsets(n), both.lens, T=int(n.sum()))
    # (the oracle's search for a page's users is quadratic: no page is shared here)
    free = iter(np.nonzero(both.ref.refs == 0)[0])
    for b in range(nseq):
        for j in range(-(-int(n[b]) // page)):
            both.ref.table[b, j] = next(free)
    both.ref.refs[both.ref.table[both.ref.table >= 0]] = 1
    assert np.array_equal(both.pool.page_table.cpu().numpy(), both.ref.table)
    assert np.array_equal(both.pool.refs.cpu().numpy(), both.ref.refs)
    before = [x.cpu().numpy() for x in _arrays(both.cache)]
    live = both.pool.compact()
    used = both.ref.refs > 0
    assert int(live.item()) == used.sum()
    to = np.arange(pages)
    src = np.nonzero(used & (to >= used.sum()))[0]
    dst = np.nonzero(~used & (to < used.sum()))[0]
    to[src] = dst
    t = both.ref.table
    assert np.array_equal(both.pool.page_table.cpu().numpy(), np.where(t >= 0, to[t], -1))
    got = both.pool.refs.cpu().numpy()
    assert (got[:used.sum()] == 1).all() and (got[used.sum():] == 0).all()
    for x, y in zip(_arrays(both.cache), before):
        y[dst] = y[src]
        assert np.array_equal(x.cpu().numpy(), y)
    both.pool.check_status()


def test_entries_outside_the_table(lib):
    """Sequences and pages that are not there are reported and left alone, positions
    outside a row too; of entries with the same child the last counts."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(8)
    both = Both(fl, rng, 12, 32, 1, 64, 4, 3)
    both.append(rng, [50, 20, 0, 0])
    both.pool.fork(i32([0, 4, 1 << 30]), i32([4, 2, 3]), both.lens)
    assert int(both.pool.status.item()) == fl.DEV_BAD_PAGE
    both.check()
    both.pool.status.zero_()
    both.pool.fork(i32([0, 1, 0]), i32([2, 2, -1]), both.lens)
    both.ref.fork([1], [2], both.n)
    both.check()
    both.pool.check_status()
    # sequence 0 would leave its row, 3 stands before its first position: only 1 is served
    both.pool.reserve(offsets([47, 15, 0, 1]), i32([50, 20, 0, -2]))
    assert int(both.pool.status.item()) == fl.DEV_BAD_PAGE
    assert both.ref.reserve([0, 15, 0, 0], both.n)
    both.check()
    both.pool.status.zero_()
    both.pool.page_table[3, 0] = 12  # no such page
    both.pool.reserve(offsets([0, 0, 0, 5]), i32([0, 0, 0, 0]))
    assert int(both.pool.status.item()) == fl.DEV_BAD_PAGE
    assert int(both.pool.page_table[3, 0].item()) == 12
    both.pool.page_table[3, 0] = -1
    both.check()


def test_padded_and_malformed_offsets(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(9)
    both = Both(fl, rng, 30, 32, 1, 64, 3, 8)
    both.pool.reserve(i32([0, 10, 10, 45]), both.lens, T=200)  # (more room than tokens)
    assert both.ref.reserve([10, 0, 35], both.n)
    both.check()
    both.pool.check_status()
    both.pool.reserve(i32([0, 200, 0, 200]), both.lens, T=200)
    assert int(both.pool.status.item()) & fl.DEV_BAD_SEQLENS
    t = both.pool.page_table.cpu().numpy()
    assert np.array_equal(np.bincount(t[t >= 0], minlength=30), both.pool.refs.cpu().numpy())


def test_captured_calls(lib):
    """A step's books captured once and replayed: fork, reserve, compact."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(10)
    both = Both(fl, rng, 60, 32, 2, 64, 5, 8)
    both.append(rng, [40, 70, 0, 0, 0])
    parents, children = i32([0, 1, 0]), i32([2, 3, 4])
    cu, lens = offsets([0, 0, 1, 1, 1]), both.lens
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both.pool.fork(parents, children, lens)
            both.pool.reserve(cu, lens)
            live = both.pool.compact()
    torch.cuda.current_stream().wait_stream(side)
    both.check()  # (nothing has run)
    for p, c in (([0, 1, 0], [2, 3, 4]), ([1, -1, 0], [2, 3, 0]), ([2, 2, 1], [3, 4, 2])):
        parents.copy_(i32(p))
        children.copy_(i32(c))
        g.replay()
        both.ref.fork(p, c, both.n)
        # (a sequence of length 0 gets its first page)
        assert both.ref.reserve([0, 0, 1, 1, 1], both.n)
        assert int(live.item()) == both.ref.compact()
        both.check()
    both.pool.check_status()
