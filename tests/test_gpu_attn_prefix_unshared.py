"""A shared prefix of which no sequence can read the pages for the others."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, bf16, i32, offsets
from tests.test_gpu_attn_prefix import Forked, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nseq,H,d", [(3, 2, 64), (3, 8, 128), (6, 16, 64)])
def test_positions_outside_the_row_are_the_plain_call_s(lib, nseq, H, d):
    """The only sequences behind the prefix stand behind their table rows: they are reported
    and get what the plain call gives them, whatever an earlier call left in the workspace."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(H)
    prefix, n = 300, [1] * nseq
    pair = Forked(fl, rng, prefix, [5 + 9 * b for b in range(nseq)], 64, 1, d)
    for x, unwritten in ((pair.gpu.k_codes, 0x7F), (pair.gpu.v_codes, 0x7F),
                         (pair.gpu.k_scales, 0xFE), (pair.gpu.v_scales, 0xFE)):
        x[x == unwritten] = 0  # (seen by sequences that stand behind all of their pages)
    q = bf16(rng, (nseq, H, d)).to(DEV)
    flags = fl.FLAG_PREFIX_ALWAYS
    size = fl.flamia_attn_cache_prefix_workspace_bytes(nseq, nseq, H, 1, d, prefix, flags)
    assert size != fl.flamia_attn_cache_workspace_bytes(nseq, nseq, H, 1, d)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)

    def run(starts, **kw):
        pair.status.zero_()
        o, lse = pair.gpu.attend(q, offsets(n), i32(starts), pair.table, d ** -0.5,
                                 dev_status=pair.status, **kw)
        return o, lse, int(pair.status.item())

    shared = dict(prefix=prefix, always_share=True)
    far = 64 * pair.t.shape[1]
    starts = [100 + b for b in range(nseq - 2)] + [far, far + 700]
    fresh = run(starts, ws=ws, **shared)
    o, lse, st = run([x - 1 for x in pair.lens], ws=ws, **shared)  # all share: parts of a prefix
    assert st == 0
    _check(o, lse, pair, q, n, [x - 1 for x in pair.lens], d ** -0.5)
    used = run(starts, ws=ws, **shared)
    plain = run(starts)
    assert fresh[2] == used[2] == plain[2] == fl.DEV_BAD_PAGE
    assert torch.isfinite(plain[0]).all() and torch.isfinite(plain[1]).all()
    assert torch.equal(fresh[0], used[0]) and torch.equal(fresh[1], used[1])
    v = max(np.abs(pair.v.values(b)).max() for b in range(nseq))
    # (BF16 outputs of either call, half a step each; weights to 2^-11)
    assert (used[0].double() - plain[0].double()).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -10) * v
    assert (used[1] - plain[1]).abs().max() <= 2.0 ** -9
    m = nseq - 2
    _check(used[0][:m], used[1][:, :m], pair, q[:m], n[:m], starts[:m], d ** -0.5)
