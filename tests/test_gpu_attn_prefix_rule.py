"""A shared prefix as the sizes decide whether it is read once: both sides of the limits, against
the oracle; and prefixes that end with a tile, read by tokens at their very end."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, bf16, i32, offsets
from tests.test_gpu_attn_prefix import Forked, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nseq,H,H_kv,d,prefix,shared", [
    # bytes saved below and above 10 MB with 8 rows of a K / V head, 20 with 16, 100 with 32
    (8, 16, 16, 128, 383, False), (8, 16, 16, 128, 384, True),
    (16, 8, 8, 64, 1407, False), (16, 8, 8, 64, 1409, True),
    (32, 16, 16, 64, 1663, False), (32, 16, 16, 64, 1664, True),
    # 300 MB with more
    (40, 32, 16, 64, 3711, False), (40, 32, 16, 64, 3712, True)])
def test_both_sides_of_the_rule(lib, nseq, H, H_kv, d, prefix, shared):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(prefix)
    size = fl.flamia_attn_cache_prefix_workspace_bytes(nseq, nseq, H, H_kv, d, prefix)
    assert (size != fl.flamia_attn_cache_workspace_bytes(nseq, nseq, H, H_kv, d)) == shared
    # (three sequences are written; the others repeat them)
    pair = Forked(fl, rng, prefix, [70, 1, 150], 64, H_kv, d)
    rows = [b % 3 for b in range(nseq)]
    pair.t = pair.t[rows]
    pair.table = torch.from_numpy(pair.t).to(DEV)
    for c in (pair.k, pair.v):
        c.codes, c.scales = [c.codes[b] for b in rows], [c.scales[b] for b in rows]
    n = [1] * nseq
    starts = [pair.lens[b] - 1 for b in rows]
    if shared:
        pair.share(n, starts)
    q = bf16(rng, (nseq, H, d)).to(DEV)
    args = q, offsets(n), i32(starts), pair.table, d ** -0.5
    o, lse = pair.gpu.attend(*args, prefix=prefix, dev_status=pair.status)
    assert pair.status.item() == 0
    _check(o, lse, pair, q, n, starts, d ** -0.5)
    if not shared:
        a = pair.gpu.attend(*args)
        assert torch.equal(o, a[0]) and torch.equal(lse, a[1])


@pytest.mark.parametrize("H,H_kv,d,nseq", [(2, 2, 64, 3), (8, 2, 128, 5), (8, 1, 64, 4), (16, 2, 128, 9),
                                           (8, 1, 64, 33)])
@pytest.mark.parametrize("prefix", [128, 384])
def test_tokens_at_the_end_of_whole_tiles(lib, H, H_kv, d, nseq, prefix):
    """A new token at prefix - 1 has no tile behind the prefix at all, one at prefix a tile of
    its own; two tokens that begin at prefix - 1 have both."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(H + prefix)
    own = [1 + b % 4 for b in range(nseq)]
    n = [2 if b % 3 == 2 else 1 for b in range(nseq)]
    starts = [prefix - 1 + (b % 3 == 1) for b in range(nseq)]
    pair = Forked(fl, rng, prefix, own, 64, H_kv, d)
    pair.share(n, starts)
    q, o, lse, scale = _run(fl, pair, rng, H, n, starts, prefix)
    assert pair.status.item() == 0
    _check(o, lse, pair, q, n, starts, scale)
    # all at prefix - 1: nobody has a tile behind it
    n, starts = [1] * nseq, [prefix - 1] * nseq
    q, o, lse, scale = _run(fl, pair, rng, H, n, starts, prefix)
    assert pair.status.item() == 0
    _check(o, lse, pair, q, n, starts, scale)
