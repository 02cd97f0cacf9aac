"""The operators together, as they are used: a prompt is written once, continuations are
forked off it, and decode steps turn, write and attend with the pool's pages over the shared
prefix; positions with axes in training and serving; captured steps."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.serving_helpers import DEV, bf16, i32, offsets
from tests.test_gpu_attn_prefix import _check

pytestmark = pytest.mark.gpu


class _Held:
    """What _check wants to know of a cache: the oracle's K and V, the GPU's head count."""

    def __init__(self, cache, k, v):
        self.gpu, self.k, self.v = cache, k, v


def _fork_oracle(held, parents, children):
    for c in (held.k, held.v):
        codes, scales = list(c.codes), list(c.scales)
        for p, b in zip(parents, children):
            c.codes[b], c.scales[b] = codes[p].copy(), scales[p].copy()


@pytest.mark.parametrize("page,H,H_kv,d,prompt,branches,axes", [(32, 4, 2, 64, 300, 5, True),
                                                                (64, 16, 2, 128, 517, 14, False),
                                                                (128, 2, 1, 128, 256, 3, True)])
def test_answers_to_one_prompt(lib, page, H, H_kv, d, prompt, branches, axes):
    """A prompt; its continuations forked and decoded; two of them forked again; one ended;
    the pool made compact in between."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(prompt)
    nseq = branches + 3
    cache = fl.KVCache(6 * nseq + prompt // page + 7, page, H_kv, d)
    cache.k_scales.fill_(0xFE)
    cache.k_codes.fill_(0x7F)
    cache.v_codes.fill_(0x7F)
    pool = fl.PagePool(cache, nseq, prompt // page + 6)
    held = _Held(cache, S.Cache(nseq, H_kv, d), S.Cache(nseq, H_kv, d))
    w = fl.rope_frequencies(d)
    rope = fl.Rotary(w, axes=fl.rope_axes([d // 8, d // 8, d // 4])) if axes else fl.Rotary(w)
    lens = torch.zeros(nseq, dtype=torch.int32, device=DEV)
    n_held = np.zeros(nseq, dtype=int)

    def step(n, prefix):
        T = sum(n)
        call = fl.DecodeCall(cache, T + 2, nseq, H, d ** -0.5, rope=rope, pool=pool, prefix=prefix,
                             always_share=True)
        q, k, v = (bf16(rng, (T + 2, h, d)).to(DEV) for h in (H, H_kv, H_kv))
        pos = i32(rng.integers(0, 4000, (3 * (T + 2)))).view(3, T + 2) if axes else None
        starts = [int(x) for x in n_held]
        o = call(q, k, v, offsets(n), lens, positions=pos)
        call.check_status()
        if axes:
            ref = S.rope_axes(q[:T].double().cpu().numpy(), pos[:, :T].cpu().numpy(), fl.rope_axes([d // 8, d // 8, d // 4]),
                              w.numpy())
            assert np.abs(call.q[:T].double().cpu().numpy() - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
        at = 0
        for b, c in enumerate(n):
            if c:
                held.k.write(b, call.k[at:at + c].double().cpu().numpy(), starts[b])
                held.v.write(b, v[at:at + c].double().cpu().numpy(), starts[b])
            at += c
        n_held[:] += n
        lens.add_(i32(n))
        _check(o[:T], call.lse[:, :T], held, call.q[:T], n, starts, d ** -0.5)
        table = pool.page_table.cpu().numpy()
        used = np.bincount(table[table >= 0], minlength=cache.num_pages)
        assert np.array_equal(used, pool.refs.cpu().numpy())

    def fork(parents, children):
        pool.fork(i32(parents), i32(children), lens)
        n_held[children] = n_held[parents]
        _fork_oracle(held, parents, children)
        assert lens.tolist() == n_held.tolist()

    step([prompt] + [0] * (nseq - 1), 0)
    pages = int((pool.refs > 0).sum())
    fork([0] * branches, list(range(1, branches + 1)))
    assert int((pool.refs > 0).sum()) == pages  # nothing copied yet
    one = [0] + [1] * branches + [0, 0]
    for _ in range(2):
        step(one, prompt)
    pool.release(i32([0, 2]), lens)
    n_held[[0, 2]] = 0
    live = pool.compact()
    assert int(live.item()) == int((pool.refs > 0).sum())
    assert (pool.refs[:int(live.item())] > 0).all()
    fork([1, 3], [nseq - 2, nseq - 1])
    step([0, 1, 0] + [2] * (branches - 2) + [1, 1], prompt)
    step([0, 1, 0] + [1] * (branches - 2) + [3, 1], prompt)


def test_captured_steps_hand_out_their_pages(lib):
    """A decode step with pages, shared prefix and axes, captured once and replayed until
    sequences cross into new pages; the same bits as eager steps."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(1)
    H, H_kv, d, page, prompt, nseq = 8, 2, 64, 32, 250, 6
    rope = fl.Rotary(fl.rope_frequencies(d), axes=fl.rope_axes([16, 16], cyclic=True))

    def build():
        cache = fl.KVCache(60, page, H_kv, d)
        pool = fl.PagePool(cache, nseq, 12)
        lens = torch.zeros(nseq, dtype=torch.int32, device=DEV)
        x = bf16(np.random.default_rng(2), (prompt, H_kv, d)).to(DEV)
        pool.reserve(offsets([prompt] + [0] * (nseq - 1)), lens)
        cache.write(x, x, offsets([prompt] + [0] * (nseq - 1)), lens, pool.page_table)
        lens[0] = prompt
        pool.fork(i32([0] * (nseq - 1)), i32(range(1, nseq)), lens)
        return cache, pool, lens, fl.DecodeCall(cache, nseq, nseq, H, d ** -0.5, rope=rope, pool=pool,
                                                    prefix=prompt, always_share=True)

    cu = offsets([1] * nseq)
    q, k, v = (torch.zeros(nseq, h, d, dtype=torch.bfloat16, device=DEV) for h in (H, H_kv, H_kv))
    pos = torch.zeros(2, nseq, dtype=torch.int32, device=DEV)
    c1, p1, l1, s1 = build()
    c2, p2, l2, s2 = build()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s1(q, k, v, cu, l1, positions=pos)
            l1.add_(1)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(40):
        for t, h in ((q, H), (k, H_kv), (v, H_kv)):
            t.copy_(bf16(rng, (nseq, h, d)))
        pos.copy_(i32(rng.integers(0, 999, 2 * nseq)).view(2, nseq))
        g.replay()
        s2(q, k, v, cu, l2, positions=pos)
        l2.add_(1)
        assert torch.equal(s1.o, s2.o) and torch.equal(s1.lse, s2.lse)
    s1.check_status()
    s2.check_status()
    assert torch.equal(p1.page_table, p2.page_table) and torch.equal(p1.refs, p2.refs)
    assert torch.equal(c1.k_codes, c2.k_codes) and torch.equal(c1.v_scales, c2.v_scales)


def test_training_call_with_axes(lib):
    """forward and backward equal the same call on turned inputs, dQ and dK turned back."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(3)
    n, H, H_kv, d = [140, 61], 4, 2, 64
    T = sum(n)
    q, do = (bf16(rng, (T, H, d)).to(DEV) for _ in range(2))
    k, v = (bf16(rng, (T, H_kv, d)).to(DEV) for _ in range(2))
    cu = offsets(n)
    pos = i32(rng.integers(0, 500, 3 * T)).view(3, T)
    rot = fl.Rotary(fl.rope_frequencies(48), interleaved=True, axes=fl.rope_axes([10, 7, 7], cyclic=True))
    call = fl.TrainingCall(T, H, d, cu, d ** -0.5, H_kv=H_kv, rope=rot, deterministic_dq=True)
    plain = fl.TrainingCall(T, H, d, cu, d ** -0.5, H_kv=H_kv, deterministic_dq=True)
    dq, dk, dv = call(q, k, v, do, positions=pos)
    call.check_status()
    qr, kr = rot(q, k, cu, positions=pos)
    o2, lse2 = plain.forward(qr, kr, v)
    dq2, dk2, dv2 = plain.backward(do)
    assert torch.equal(call.o, o2) and torch.equal(call.lse, lse2) and torch.equal(dv, dv2)
    dq2, dk2 = rot(dq2, dk2, cu, positions=pos, inverse=True)
    assert torch.equal(dq, dq2) and torch.equal(dk, dk2)


@pytest.mark.parametrize("far", [False, True])
def test_a_step_without_its_pages_does_nothing(lib, far):
    """Two continuations share a half-filled page.  A step for which there is no page left (or
    with a sequence behind its row) leaves pages, books and outputs as they are and says so;
    with pages it goes on from there."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(7)
    H, H_kv, d, page, prompt, nseq = 4, 2, 64, 64, 160, 3
    cache = fl.KVCache(3 if not far else 9, page, H_kv, d)
    pool = fl.PagePool(cache, nseq, 4)
    lens = torch.zeros(nseq, dtype=torch.int32, device=DEV)
    cu = offsets([prompt, 0, 0])
    pool.reserve(cu, lens)
    x = bf16(rng, (prompt, H_kv, d)).to(DEV)
    cache.write(x, x, cu, lens, pool.page_table)
    lens[0] = prompt
    pool.fork(i32([0]), i32([1]), lens)
    call = fl.DecodeCall(cache, 3, nseq, H, d ** -0.5, rope=fl.Rotary(fl.rope_frequencies(d)), pool=pool)
    cu = offsets([1, 1, 1])
    starts = lens.clone()
    if far:
        starts[2] = 4 * page
    else:
        cu[3] = 2
    q, k, v = (bf16(rng, (3, h, d), 50.0).to(DEV) for h in (H, H_kv, H_kv))
    call.o.fill_(7)
    call.lse.fill_(7)
    held = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)]
    table = pool.page_table.clone()
    call(q, k, v, cu, starts)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="0x10" if far else "0x2$"):
        call.check_status()
    assert (call.o == 7).all() and (call.lse == 7).all() and (call.granted == 0).all()
    if far:  # (the books keep what the others took)
        assert torch.equal(pool.page_table[2], table[2])
        assert set(pool.page_table[:2].flatten().tolist()) == set(table[0].tolist()) | {3}
    else:
        assert torch.equal(pool.page_table, table)
        assert all(map(torch.equal, held, (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)))
    # one of the two alone has pages enough, after the other has gone
    pool.release(i32([1]), lens)
    pool.status.zero_()
    call(q, k, v, offsets([1, 0, 0]), lens)
    call.check_status()
    assert torch.equal(call.granted, offsets([1, 0, 0]))
    assert (call.o[0] != 7).any() and (call.o[1:] == 7).all()
