"""The operators together, as they are used: a prompt and decode steps through
rotary positions, cache and attention; rotary positions inside the training
call; captured steps."""
import numpy as np
import pytest
import torch

from oracle import flamia_oracle as O
from oracle import serving_oracle as S
from tests.gpu_helpers import compare
from tests.serving_helpers import DEV, Pair, bf16, check_attend, i32, offsets, page_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_prompt_then_single_tokens(lib, window, sinks):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(31)
    H, H_kv, d, nseq = 4, 2, 64, 3
    steps = [[70, 5, 0], [1, 1, 33], [1, 0, 1], [1, 4, 1], [1, 1, 1]]
    pair = Pair(fl, rng, np.sum(steps, axis=0), 32, H_kv, d)
    rot = fl.Rotary(fl.rope_frequencies(d))
    lens = np.zeros(nseq, dtype=int)
    for n in steps:
        T = sum(n)
        step = fl.DecodeCall(pair.gpu, T, nseq, H, d ** -0.5, rope=rot, window=window, sinks=sinks)
        q, k, v = (bf16(rng, (T, h, d)).to(DEV) for h in (H, H_kv, H_kv))
        starts = [int(x) for x in lens]
        o = step(q, k, v, offsets(n), i32(starts), pair.table)
        step.check_status()
        # the oracle takes the rotated BF16 rows that the cache was given
        at = 0
        for b, c in enumerate(n):
            if c:
                pair.k.write(b, step.k[at:at + c].double().cpu().numpy(), starts[b])
                pair.v.write(b, v[at:at + c].double().cpu().numpy(), starts[b])
            at += c
        lens += n
        pair.check_equal(lens)
        check_attend(o, step.lse, pair, step.q, n, starts, d ** -0.5, window, sinks)
        pos = np.concatenate([np.arange(s, s + c) for s, c in zip(starts, n)])
        ref = S.rope(q.double().cpu().numpy(), pos, fl.rope_frequencies(d).numpy())
        assert np.abs(step.q.double().cpu().numpy() - ref).max() <= (2.0 ** -8 + 2.0 ** -18) * np.abs(ref).max()


def test_cached_attention_agrees_with_the_training_forward(lib):
    """A prompt's cached attention (BF16 queries, unrounded weights) against the
    training forward (E4M3 queries and weights) on the same K and V codes."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(32)
    n, H, d = [200, 57], 4, 128
    T = sum(n)
    q, k, v = (bf16(rng, (T, H, d)).to(DEV) for _ in range(3))
    cu = offsets(n)
    call = fl.TrainingCall(T, H, d, cu, d ** -0.5)
    o, lse = call.forward(q, k, v)
    t, pages = page_table(rng, n, 128)
    cache = fl.KVCache(pages, 128, H, d)
    table = torch.from_numpy(t).to(DEV)
    cache.write(k, v, cu, None, table)
    o2, lse2 = cache.attend(q, cu, None, table, d ** -0.5)
    compare("o", o2.double().cpu().numpy(), o.double().cpu().numpy(), 0.998, 6e-2)
    assert (lse - lse2).abs().max() < 0.1


def test_training_call_with_rotary_positions(lib):
    """forward and backward with rope equal the same call on rotated inputs, dQ and
    dK turned back, and agree with the float64 gradient of the whole."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(33)
    n, H, H_kv, d = [140, 61], 4, 2, 64
    T = sum(n)
    q, do = (bf16(rng, (T, H, d)).to(DEV) for _ in range(2))
    k, v = (bf16(rng, (T, H_kv, d)).to(DEV) for _ in range(2))
    cu = offsets(n)
    rot = fl.Rotary(fl.rope_frequencies(48, factor=2.0), interleaved=True)
    call = fl.TrainingCall(T, H, d, cu, d ** -0.5, H_kv=H_kv, rope=rot, deterministic_dq=True)
    plain = fl.TrainingCall(T, H, d, cu, d ** -0.5, H_kv=H_kv, deterministic_dq=True)
    keep = q.clone(), k.clone()
    o, lse = call.forward(q, k, v)
    dq, dk, dv = call.backward(do)
    call.check_status()
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])
    qr, kr = rot(q, k, cu)
    o2, lse2 = plain.forward(qr, kr, v)
    dq2, dk2, dv2 = plain.backward(do)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(dv, dv2)
    dq2, dk2 = rot(dq2, dk2, cu, inverse=True)
    assert torch.equal(dq, dq2) and torch.equal(dk, dk2)
    # unquantised float64 attention of rotated rows, gradients turned back
    pos = np.concatenate([np.arange(c) for c in n])
    w = fl.rope_frequencies(48, factor=2.0).numpy()
    f = lambda t: t.double().cpu().numpy()
    ref = O.attention(S.rope(f(q), pos, w, True), S.rope(f(k), pos, w, True), f(v), f(do),
                      [0, 140, 201], d ** -0.5, quant=False)
    compare("dq", f(dq), S.rope(ref["dQ"], pos, w, True, inverse=True), 0.99, 0.2)
    compare("dk", f(dk), S.rope(ref["dK"], pos, w, True, inverse=True), 0.99, 0.2)


def test_captured_step_is_replayed_on_new_positions(lib):
    """One decode step captured once and replayed while tokens, positions and page
    table change in place; two captured steps share a cache and a workspace."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(34)
    H, H_kv, d, nseq, steps = 8, 2, 128, 4, 6
    first = [30, 0, 65, 200]
    pair = Pair(fl, rng, [f + steps for f in first], 32, H_kv, d)
    x = bf16(rng, (sum(first), H_kv, d))
    pair.write(x, x, first, [0] * nseq)
    rot = fl.Rotary(fl.rope_frequencies(d))
    call = fl.DecodeCall(pair.gpu, nseq, nseq, H, d ** -0.5, rope=rot)
    cu, starts = offsets([1] * nseq), i32(first)
    q, k, v = (torch.zeros(nseq, h, d, dtype=torch.bfloat16, device=DEV) for h in (H, H_kv, H_kv))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call(q, k, v, cu, starts, pair.table)
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    lens = list(first)
    for i in range(steps):
        for t, h in ((q, H), (k, H_kv), (v, H_kv)):
            t.copy_(bf16(rng, (nseq, h, d)))
        starts.copy_(i32(lens))
        graphs[i % 2].replay()
        call.check_status()
        for b in range(nseq):
            pair.k.write(b, call.k[b:b + 1].double().cpu().numpy(), lens[b])
            pair.v.write(b, v[b:b + 1].double().cpu().numpy(), lens[b])
        check_attend(call.o, call.lse, pair, call.q, [1] * nseq, lens, d ** -0.5)
        lens = [x + 1 for x in lens]
        pair.check_equal(lens)
