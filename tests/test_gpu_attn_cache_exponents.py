"""Attention over the paged cache where scores and value exponents change along a
sequence by far more than float32 could hold at once, in every row form (8, 16, 32
and 256 query rows an item)."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.serving_helpers import (DEV, Pair, attend_tolerance, bf16, check_attend, i32, lse_tolerance,
                                   offsets, weight_error)

pytestmark = pytest.mark.gpu

# (x, eV) of the 128-key tiles: scores 2^x, values near 2^eV
TILES = {
    # every tile adds the same to the output, the first holds the softmax's weight
    "values climb as scores fall": [(-32 * t, 32 * t - 100) for t in range(7)],
    "by steps that do not move the exponent": [(-24 * t, 24 * t - 100) for t in range(8)],
    "by large steps": [(-96 * t, 96 * t - 110) for t in range(3)] + [(-192, 82)] * 3,
    # and back: the references move while the exponent of the sums lags behind
    "then scores return": [(-32 * t, 32 * t - 100) for t in range(5)] + [(20, 30), (-40, 60)],
    "then values return": [(-40 * t, 40 * t - 100) for t in range(5)] + [(0, -100), (48, -100)],
    "values fall as scores climb": [(32 * t, 90 - 32 * t) for t in range(7)],
    "up and down": [(0, 60), (60, -90), (-60, 90), (100, -100), (-100, 100), (0, 0), (40, 20)],
}

# new tokens, H, H_kv, d, sequences, rows an item
FORMS = [(1, 2, 2, 128, 400, 8), (1, 4, 1, 64, 700, 8), (6, 4, 2, 128, 300, 16),
         (5, 6, 2, 64, 300, 16), (40, 2, 2, 128, 150, 32), (20, 4, 1, 64, 300, 32),
         (140, 2, 2, 128, 200, 256), (50, 4, 1, 64, 300, 256)]


def largest_weight(q, k, start, scale, e, window=0):
    """[n, H] of queries q at positions start ..: the largest p 448 2^e of a seen key,
    which bounds what a weight below the range may lose (no exponent is cut off)."""
    n, H, _ = q.shape
    out = np.zeros((n, H))
    for i in range(n):
        m = S.seen_keys(start + i, len(k), window)
        for h in range(H):
            x = k[m, h * k.shape[1] // H] @ q[i, h] * scale
            lse = x.max() + np.log(np.exp(x - x.max()).sum())
            out[i, h] = 448 * np.exp2(((x - lse) / np.log(2) + e[m, h * k.shape[1] // H]).max())
    return out


def test_forms_take_their_rows():
    """The rule on the mean number of rows, as the forms above expect it."""
    for n, H, H_kv, _, _, want in FORMS:
        rows = n * (H // H_kv)
        assert want == (8 if rows <= 8 else 16 if rows <= 16 else 32 if rows <= 96 else 256)


@pytest.mark.parametrize("name", sorted(TILES))
@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("n,H,H_kv,d,nseq,rows", FORMS)
def test_scores_and_value_exponents_that_move_apart(lib, name, n, H, H_kv, d, nseq, rows, token):
    """The same sequence many times over the same pages, so that every CTA has a run
    of several items and most of them whole, against float64."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(len(name) + n + d)
    tiles = TILES[name]
    L = 128 * len(tiles)
    x = torch.tensor([t[0] for t in tiles], dtype=torch.float64).repeat_interleave(128)
    e = torch.tensor([t[1] for t in tiles], dtype=torch.float64).repeat_interleave(128)
    k = bf16(rng, (L, H_kv, d), 0.05)
    k[:, :, 0] = x[:, None].to(torch.bfloat16)
    v = (bf16(rng, (L, H_kv, d)).double() * torch.exp2(e)[:, None, None]).to(torch.bfloat16)
    pair = Pair(fl, rng, [L], 128, H_kv, d, token)
    pair.write(k, v, [L], [0])
    q1 = bf16(rng, (n, H, d), 0.05)
    q1[:, :, 0] = d ** 0.5 * float(np.log(2.0))
    table = pair.table.expand(nseq, -1).contiguous()
    q = q1.repeat(nseq, 1, 1).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = pair.gpu.attend(q, offsets([n] * nseq), i32([L - n] * nseq), table, d ** -0.5,
                             dev_status=st)
    assert int(st.item()) == 0
    qn, kn, vn = q1.double().numpy(), pair.k.values(0), pair.v.values(0)
    e = pair.v.scales[0].astype(int) - 127
    ro, rl, mass, _ = S.attend(qn, kn, vn, L - n, d ** -0.5, v_exponents=e)
    top = largest_weight(qn, kn, L - n, d ** -0.5, e)
    tol = attend_tolerance(qn, kn, d ** -0.5, L, ro, weight_error(n, 1, H // H_kv), mass,
                           top[..., None])
    got = o.view(nseq, n, H, d).double().cpu().numpy()
    gl = lse.view(H, nseq, n).double().cpu().numpy()
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    err = np.abs(got - ro[None]) / np.maximum(tol, 2.0 ** -133)
    assert err.max() <= 1, ("o", err.max(), int((err.reshape(nseq, -1).max(1) > 1).sum()))
    err = np.abs(gl - rl[:, None]) / lse_tolerance(qn, kn, d ** -0.5, rl)[:, None]
    assert err.max() <= 1, ("lse", err.max())


UNSEEN = [
    # where the huge values lie (positions from the end of the context) and the window
    ("the last draft", lambda n: [0], 0),
    ("the second half of the drafts", lambda n: range(n // 2), 0),
    ("keys that only the first draft sees", lambda n: [n - 1 + 199], 200),
    ("keys behind the window and one inside", lambda n: [n + 199, n + 400, 3], 200),
]


@pytest.mark.parametrize("where,at,window", UNSEEN, ids=[u[0] for u in UNSEEN])
@pytest.mark.parametrize("large", [2.0 ** 70, 2.0 ** 100])
@pytest.mark.parametrize("n,H,H_kv,d,nseq,rows", [(2, 4, 1, 128, 3, 8), (4, 2, 1, 64, 3, 8),
                                                  (6, 4, 2, 128, 3, 16), (40, 2, 2, 64, 2, 32),
                                                  (140, 2, 2, 128, 2, 256), (60, 4, 1, 64, 2, 256)])
def test_a_large_value_that_a_row_does_not_see(lib, where, at, window, large, n, H, H_kv, d, nseq,
                                               rows):
    """Rows that do not see it are what they are without it: the exponents that rows
    side by side have in common must not cost one of them its values."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(n + d)
    L = 700
    pair = Pair(fl, rng, [L] * nseq, 64, H_kv, d, True)  # (a token has an exponent of its own)
    k, v = (bf16(rng, (nseq * L, H_kv, d)) for _ in range(2))
    for b in range(nseq):
        for p in at(n):
            v[b * L + L - 1 - p] = (v[b * L + L - 1 - p].double() * large).to(torch.bfloat16)
    pair.write(k, v, [L] * nseq, [0] * nseq)
    q = bf16(rng, (nseq * n, H, d)).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = pair.gpu.attend(q, offsets([n] * nseq), i32([L - n] * nseq), pair.table, d ** -0.5,
                             window=window, dev_status=st)
    assert int(st.item()) == 0
    check_attend(o, lse, pair, q, [n] * nseq, [L - n] * nseq, d ** -0.5, window)
    for b in range(nseq):  # (and by the bound of the row's own keys)
        qn, kn, vn = q[b * n:b * n + n].double().cpu().numpy(), pair.k.values(b), pair.v.values(b)
        e = pair.v.scales[b].astype(int) - 127
        ro, _, mass, _ = S.attend(qn, kn, vn, L - n, d ** -0.5, window, 0, e)
        top = largest_weight(qn, kn, L - n, d ** -0.5, e, window)
        tol = attend_tolerance(qn, kn, d ** -0.5, L, ro, weight_error(nseq * n, nseq, H // H_kv), mass,
                               top[..., None])
        err = np.abs(o[b * n:b * n + n].double().cpu().numpy() - ro) / np.maximum(tol, 2.0 ** -133)
        assert err.max() <= 1, (b, err.max())
