"""Steps whose kernels overlap (programmatic dependent launch, replayed graphs)
against the same calls with the device idle between any two kernels, bit for bit."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, bf16, i32, offsets, page_table

pytestmark = pytest.mark.gpu

STEPS = [
    # new tokens, first starts, H, H_kv, d, page: chunks of more than 96 rows, drafts and
    # single tokens that begin inside a 32-token block
    ([140, 101], [37, 1003], 2, 2, 128, 64),
    ([50, 33, 60], [5, 511, 290], 8, 2, 64, 32),
    ([3, 2, 4, 1], [29, 63, 700, 2049], 8, 2, 128, 128),
    ([1] * 9, [30 + 97 * i for i in range(9)], 4, 4, 64, 64),
]


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("n,first,H,H_kv,d,page", STEPS)
def test_replayed_steps(lib, n, first, H, H_kv, d, page, token):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(sum(n) + d)
    nseq, T, rounds = len(n), sum(n), 25
    t, pages = page_table(rng, [f + c + rounds for f, c in zip(first, n)], page)
    table = torch.from_numpy(t).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(T)
    rows = lambda m, h: torch.randn(m, h, d, generator=g, device=DEV).to(torch.bfloat16)
    caches = [fl.KVCache(pages, page, H_kv, d, token_scales=token) for _ in range(2)]
    k0, v0 = rows(sum(first), H_kv), rows(sum(first), H_kv)
    for c in caches:
        c.write(k0, v0, offsets(first), None, table)
    rot = fl.Rotary(fl.rope_frequencies(d))
    step = fl.DecodeCall(caches[0], T, nseq, H, d ** -0.5, rope=rot)
    cu, starts = offsets(n), i32(first)
    q, k, v = rows(T, H), rows(T, H_kv), rows(T, H_kv)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q, k, v, cu, starts, table)
    for i in range(rounds):
        # (one token further each time: the chunk before is partly written again)
        for x, h in ((q, H), (k, H_kv), (v, H_kv)):
            x.copy_(rows(T, h))
        starts.copy_(i32([f + i for f in first]))
        graph.replay()
        want = caches[1]
        torch.cuda.synchronize()
        qr, kr = rot(q, k, cu, starts)
        torch.cuda.synchronize()
        want.write(kr, v, cu, starts, table)
        torch.cuda.synchronize()
        o, lse = want.attend(qr, cu, starts, table, d ** -0.5)
        torch.cuda.synchronize()
        assert torch.equal(step.o, o) and torch.equal(step.lse, lse), i
        for a, b in ((caches[0].k_codes, want.k_codes), (caches[0].v_codes, want.v_codes),
                     (caches[0].k_scales, want.k_scales), (caches[0].v_scales, want.v_scales)):
            assert torch.equal(a, b), i
    step.check_status()


def test_beside_a_training_call(lib):
    """Decode steps and prompts on two streams while a third trains: each gives the bits
    that it gives alone (the kernels share the SMs' tensor memory, nothing else)."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(91)
    d, H, H_kv, T = 128, 8, 2, 1500
    cu = offsets([1000, 500])
    x = [bf16(rng, (T, h, d)).to(DEV) for h in (H, H_kv, H_kv, H)]
    rot = fl.Rotary(fl.rope_frequencies(d))
    train = fl.TrainingCall(T, H, d, cu, d ** -0.5, H_kv=H_kv, deterministic_dq=True, rope=rot)
    jobs = []
    for n, first in (([1] * 40, 1200), ([300, 211], 700)):
        nseq, m = len(n), sum(n)
        t, pages = page_table(rng, [first + c for c in n], 64)
        cache = fl.KVCache(pages, 64, H_kv, d)
        table = torch.from_numpy(t).to(DEV)
        k, v = (bf16(rng, (first * nseq, H_kv, d)).to(DEV) for _ in range(2))
        cache.write(k, v, offsets([first] * nseq), None, table)
        step = fl.DecodeCall(cache, m, nseq, H, d ** -0.5, rope=rot)
        args = ([bf16(rng, (m, h, d)).to(DEV) for h in (H, H_kv, H_kv)] +
                [offsets(n), i32([first] * nseq), table])
        jobs.append((step, args))
    want = [[y.clone() for y in train(*x)] + [train.o.clone()]]
    for step, args in jobs:
        step(*args)
        want.append([step.o.clone(), step.lse.clone()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(12):
        with torch.cuda.stream(streams[0]):
            train(*x)
        for s, (step, args) in zip(streams[1:], jobs):
            with torch.cuda.stream(s):
                for _ in range(4):
                    step(*args)
    torch.cuda.synchronize()
    got = [[train.dq, train.dk, train.dv, train.o]] + [[step.o, step.lse] for step, _ in jobs]
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    train.check_status()
    for step, _ in jobs:
        step.check_status()
