"""Rotary positions on the GPU against float64."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.serving_helpers import DEV, bf16, i32, offsets

pytestmark = pytest.mark.gpu


def _check(got, x, pos, w, inter, mscale, inverse):
    """BF16 rounding is half a step, 2^-8 of the value.  The angle is off by
    2 pi 2^-32 (its top 32 bits) and pi 2^-24 (as float32), sine and cosine by
    2^-22, the products and the sum by 3 * 2^-24: below 2^-20 of the pair."""
    x = x.double().cpu().numpy()
    ref = S.rope(x, pos, w, inter, mscale, inverse)
    r = 2 * len(w)
    size = np.abs(x).copy()
    a, b = (np.arange(0, r, 2), np.arange(1, r, 2)) if inter else (np.arange(r // 2),
                                                                   np.arange(r // 2, r))
    size[..., a] = size[..., b] = size[..., a] + size[..., b]
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * mscale * size
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / tol.clip(1e-30)).max()
    assert np.array_equal(got.double().cpu().numpy()[..., r:], x[..., r:])


CASES = [
    # lengths, H, H_kv, d, rot_dim, interleaved, inverse
    ([1], 1, 1, 64, 16, False, False),
    ([1, 1, 1], 8, 2, 128, 128, False, False),
    ([5, 0, 9], 3, 3, 64, 64, True, False),
    ([5, 0, 9], 3, 1, 64, 48, False, True),
    ([700, 1, 800], 7, 5, 128, 96, True, True),
    ([2000], 16, 16, 128, 128, False, True),
    ([1300, 17], 32, 8, 64, 32, True, False),
]


@pytest.mark.parametrize("n,H,H_kv,d,r,inter,inverse", CASES)
def test_rope(lib, n, H, H_kv, d, r, inter, inverse):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(d + r + H)
    T = sum(n)
    q, k = bf16(rng, (T, H, d)).to(DEV), bf16(rng, (T, H_kv, d)).to(DEV)
    starts = [int(s) for s in rng.integers(0, 1 << 20, len(n))]
    pos = np.concatenate([np.arange(s, s + c) for s, c in zip(starts, n)])
    w = fl.rope_frequencies(r, factor=2.0)
    rot = fl.Rotary(w, interleaved=inter, mscale=1.25)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo, ko = rot(q, k, offsets(n), i32(starts), inverse=inverse, dev_status=st)
    _check(qo, q, pos, w.numpy(), inter, 1.25, inverse)
    _check(ko, k, pos, w.numpy(), inter, 1.25, inverse)
    # in place, and without K
    q2, k2 = q.clone(), k.clone()
    rot(q2, k2, offsets(n), i32(starts), q_out=q2, k_out=k2, inverse=inverse, dev_status=st)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    q3, none = rot(q, None, offsets(n), i32(starts), inverse=inverse, dev_status=st)
    assert none is None and torch.equal(q3, qo)
    assert int(st.item()) == 0


def test_slices_of_a_packed_projection(lib):
    """Q and K inside one [T, H + 2 H_kv, d] tensor, turned in place; V and the rows
    behind the last document keep their bits."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(3)
    T, H, H_kv, d = 37, 4, 2, 64
    x = bf16(rng, (T, H + 2 * H_kv, d)).to(DEV)
    before = x.clone()
    w = fl.rope_frequencies(d)
    q, k = x[:, :H], x[:, H:H + H_kv]
    fl.Rotary(w)(q, k, offsets([30, 3]), i32([5, 0]), q_out=q, k_out=k)
    pos = np.concatenate([np.arange(5, 35), np.arange(3)])
    _check(q[:33], before[:33, :H], pos, w.numpy(), False, 1.0, False)
    _check(k[:33], before[:33, H:H + H_kv], pos, w.numpy(), False, 1.0, False)
    assert torch.equal(x[:, H + H_kv:], before[:, H + H_kv:]) and torch.equal(x[33:], before[33:])


def test_far_positions_keep_their_angle(lib):
    """The slowest and the fastest pair at positions up to 2^31 - 2: the wrapped
    product holds the angle where float32 would have lost it."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(4)
    pos = [0, 1, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 2, -5]
    x = bf16(rng, (len(pos), 2, 128)).to(DEV)
    # frequencies that are whole multiples of 2^-64 turns: the table is exact
    turns = np.array([2.0 ** -1, 2.0 ** -2, 2.0 ** -10, 3 * 2.0 ** -20, 5 * 2.0 ** -33, 2.0 ** -40,
                      2.0 ** -50, 7 * 2.0 ** -60])
    rot = fl.Rotary(2 * np.pi * turns)
    rot.turns = torch.tensor([s - (1 << 64) if s >> 63 else s for s in
                              (int(t * 2.0 ** 64) for t in turns)], dtype=torch.int64, device=DEV)
    y, _ = rot(x, None, offsets([1] * len(pos)), i32(pos))
    # the oracle's angle from the exact fraction of a turn
    frac = np.array([[(p * int(t * 2.0 ** 64)) % (1 << 64) / 2.0 ** 64 for t in turns] for p in pos])
    xd = x.double().cpu().numpy()
    c, s = np.cos(2 * np.pi * frac)[:, None], np.sin(2 * np.pi * frac)[:, None]
    ref = xd.copy()
    ref[..., :8] = xd[..., :8] * c - xd[..., 8:16] * s
    ref[..., 8:16] = xd[..., :8] * s + xd[..., 8:16] * c
    size = np.abs(xd[..., :8]) + np.abs(xd[..., 8:16])
    tol = 2.0 ** -8 * np.abs(ref)
    tol[..., :16] += 2.0 ** -20 * np.concatenate([size, size], -1)
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()


def test_gradient_is_the_inverse(lib):
    """<R x, g> = <x, R^T g> up to the BF16 rounding of the two results."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(5)
    x, g = bf16(rng, (64, 4, 128)).to(DEV), bf16(rng, (64, 4, 128)).to(DEV)
    rot = fl.Rotary(fl.rope_frequencies(128), interleaved=True)
    y, _ = rot(x, None, offsets([64]))
    b, _ = rot(g, None, offsets([64]), inverse=True)
    yd, gd, xd, bd = (t.double() for t in (y, g, x, b))
    # each product is off by at most half a BF16 step (2^-8) of itself
    bound = 2.0 ** -8 * ((yd * gd).abs().sum() + (xd * bd).abs().sum()) * 1.01
    assert float(((yd * gd).sum() - (xd * bd).sum()).abs()) <= float(bound)


def test_malformed_offsets_are_reported(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    x = torch.ones(8, 2, 64, dtype=torch.bfloat16, device=DEV)
    for cu in ([0, 9], [1, 8], [0, 6, 4, 8], [0, -3, 8]):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        fl.Rotary(fl.rope_frequencies(64))(x, x, i32(cu), dev_status=st)
        assert int(st.item()) == fl.DEV_BAD_SEQLENS, cu
