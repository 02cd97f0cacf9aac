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
