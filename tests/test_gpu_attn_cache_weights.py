"""Softmax weights far below the row's largest: each output element holds one key's
weight alone, so its rounding shows."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.serving_helpers import DEV, Pair, attend_tolerance, bf16, i32, offsets, weight_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,H,H_kv,rows", [(1, 2, 2, 8), (4, 4, 2, 8), (1, 16, 1, 16), (12, 2, 2, 16),
                                           (30, 1, 1, 32), (90, 2, 2, 32), (70, 4, 2, 256)])
def test_small_weights(lib, n, H, H_kv, rows, d, token):
    """A heavy key without a value, and a key for each element of the head whose weight
    lies 2^-0.2 .. 2^-20 below it, the same for every query."""
    from precision_causal_attention_block_gb300 import flamia as fl
    mean = n * (H // H_kv)
    assert rows == (8 if mean <= 8 else 16 if mean <= 16 else 32 if mean <= 96 else 256)
    rng = np.random.default_rng(d + n)
    L = d + 1 + n  # (the queries' own keys have no value either)
    k = torch.zeros(L, H_kv, d, dtype=torch.bfloat16)
    v = torch.zeros(L, H_kv, d, dtype=torch.bfloat16)
    order = torch.from_numpy(rng.permutation(d))
    j = torch.arange(d)
    # scores in steps that E4M3 holds: several elements of the key add up
    x = 20.0 * (j + 1.0) / d
    for i in range(4):
        part = (x * 2.0 ** i * 8).floor() / (2.0 ** i * 8) if i < 3 else x
        k[1 + j, :, i] = -(part[:, None]).to(torch.bfloat16)
        x = x - part
    k[d + 1:, :, 0] = -30.0
    v[1 + j, :, order] = 1.0
    pair = Pair(fl, rng, [L], 32, H_kv, d, token)
    pair.write(k, v, [L], [0])
    q = torch.zeros(n, H, d, dtype=torch.bfloat16)
    q[:, :, :4] = d ** 0.5 * float(np.log(2.0))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, _ = pair.gpu.attend(q.to(DEV), offsets([n]), i32([L - n]), pair.table, d ** -0.5, dev_status=st)
    assert int(st.item()) == 0
    qn, kn, vn = q.double().numpy(), pair.k.values(0), pair.v.values(0)
    ref, _, mass, top = S.attend(qn, kn, vn, L - n, d ** -0.5,
                                 v_exponents=pair.v.scales[0].astype(int) - 127)
    assert ref.min() < 2.0 ** -19 * ref.max()
    tol = attend_tolerance(qn, kn, d ** -0.5, 1, ref, weight_error(n, 1, H // H_kv), mass,
                           top[..., None])
    err = np.abs(o.double().cpu().numpy() - ref) / tol
    assert err.max() <= 1, (err.max(), ref.ravel()[err.argmax()])
