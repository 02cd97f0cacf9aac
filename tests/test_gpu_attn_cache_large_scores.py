"""Scores so large that float32 holds no fractions of them: the softmax is one key's
value, or a mean of those whose scores float32 cannot tell apart."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.serving_helpers import DEV, Pair, bf16, check_attend, i32, offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [12, 17, 20, 24, 28, 33, 40, 60, 90])
@pytest.mark.parametrize("n,H,H_kv,d,nseq,token", [(1, 2, 2, 64, 1, False), (3, 4, 2, 128, 40, False),
                                                   (12, 2, 2, 64, 3, True), (40, 2, 2, 128, 2, False),
                                                   (140, 2, 2, 128, 2, False), (150, 1, 1, 64, 2, True)])
def test_large_scores(lib, power, n, H, H_kv, d, nseq, token):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(power + n)
    L = 1100
    pair = Pair(fl, rng, [L], 64, H_kv, d, token)
    half = 2.0 ** (power // 2)
    pair.write(bf16(rng, (L, H_kv, d), half), bf16(rng, (L, H_kv, d)), [L], [0])
    q1 = bf16(rng, (n, H, d), 2.0 ** (power - power // 2))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = pair.gpu.attend(q1.repeat(nseq, 1, 1).to(DEV), offsets([n] * nseq), i32([L - n] * nseq),
                             pair.table.expand(nseq, -1).contiguous(), d ** -0.5, dev_status=st)
    assert int(st.item()) == 0
    q, k, v = q1.double().numpy(), pair.k.values(0), pair.v.values(0)
    got = o.view(nseq, n, H, d).double().cpu().numpy()
    gl = lse.view(H, nseq, n).double().cpu().numpy()
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    G = H // H_kv
    told = 0
    for i in range(n):
        seen = L - n + i + 1
        for h in range(H):
            x = k[:seen, h // G] @ q[i, h] * d ** -0.5
            vs = v[:seen, h // G]
            # a mean of values, whatever the scores (BF16 rounding: half a step; the sum of
            # the weights: 2^-20)
            assert (got[:, i, h] <= vs.max(0) + 2.0 ** -7 * np.abs(vs).max(0)).all()
            assert (got[:, i, h] >= vs.min(0) - 2.0 ** -7 * np.abs(vs).max(0)).all()
            # sums of d products in float32, in an order of the tensor core's own: d 2^-24 of
            # their magnitudes, on both sides; scores within 2^-19 of the reference are equal
            off = (2 * d * 2.0 ** -24 * np.abs(k[:seen, h // G] * q[i, h]).sum(1).max() * d ** -0.5
                   + 2.0 ** -18 * np.abs(x).max())
            assert (np.abs(gl[h, :, i] - x.max()) <= off + np.log(seen) + 1e-3).all()
            best = int(x.argmax())
            if np.sort(x)[-2] < x[best] - off - 20:
                told += 1
                # 2^-24 of the weights of 1,100 keys at most
                tol = 2.0 ** -8 * np.abs(vs[best]) + seen * np.exp(-20) * np.abs(vs).max()
                assert (np.abs(got[:, i, h] - vs[best]) <= tol).all(), (i, h)
    assert told > 0 or power < 20
