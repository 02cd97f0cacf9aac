"""Rotary positions with several axes against the oracle, forward and transposed."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.serving_helpers import DEV, bf16, i32, offsets

pytestmark = pytest.mark.gpu

# BF16 rounding (half a step, 2^-8 of a value of at most the row's pair norm), sine and
# cosine (2^-26 turns of angle, a few 2^-24 of float32) and two float32 products
TOL = 2.0 ** -8 + 2.0 ** -20


def _check(got, x, pos, axes, w, inter, m, inverse):
    ref = S.rope_axes(x.double().cpu().numpy(), pos, axes, w, inter, m, inverse)
    r, xx = 2 * len(w), x.double().cpu().numpy()
    a = np.arange(0, r, 2) if inter else np.arange(r // 2)
    b = a + 1 if inter else a + r // 2
    size = np.abs(xx)
    pair = m * np.hypot(xx[..., a], xx[..., b])
    size[..., a] = size[..., b] = pair
    assert (np.abs(got.double().cpu().numpy() - ref) <= TOL * size + 2.0 ** -133).all()


@pytest.mark.parametrize("T,H,H_kv,d,rot,sections,cyclic,inter,m", [
    (1, 4, 2, 64, 64, [8, 12, 12], False, False, 1.0),
    (37, 4, 1, 128, 128, [16, 24, 24], False, False, 1.0),
    (300, 2, 2, 128, 96, [20, 14, 14], True, True, 1.25),
    (455, 3, 0, 64, 16, [2, 3, 3], True, False, 1.0),
    (457, 3, 5, 64, 48, [24], False, True, 1.0),
    (1001, 8, 2, 128, 64, [1, 0, 30, 1], False, True, 0.5),
    (700, 2, 1, 128, 128, [1] * 64, False, False, 1.0),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_axes(lib, T, H, H_kv, d, rot, sections, cyclic, inter, m, inverse):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(T)
    axes = fl.rope_axes(sections, cyclic=cyclic)
    w = fl.rope_frequencies(rot)
    rope = fl.Rotary(w, interleaved=inter, mscale=m, axes=axes)
    n = len(sections)
    pos = rng.integers(-3, 200000, (n, T))
    pos[:, 0] = [2 ** 31 - 1 if a % 2 else -2 ** 31 for a in range(n)]
    q = bf16(rng, (T, H, d)).to(DEV)
    k = bf16(rng, (T, H_kv, d)).to(DEV) if H_kv else None
    p = torch.from_numpy(pos.astype(np.int32)).to(DEV)
    # frequencies as the kernel has them (turns of 2^-64), so far positions agree
    steps = np.array([int(t) % 2 ** 64 for t in rope.turns.tolist()], dtype=object)
    exact = np.array([float(s) for s in steps]) * 2 * np.pi / 2.0 ** 64
    near = np.abs(pos) <= 200000
    qo, ko = rope(q, k, offsets([T]), positions=p, inverse=inverse)
    rows = near.all(0)
    _check(qo[torch.from_numpy(rows).to(DEV)], q[torch.from_numpy(rows).to(DEV)], pos[:, rows], axes, exact,
           inter, m, inverse)
    if H_kv:
        _check(ko[torch.from_numpy(rows).to(DEV)], k[torch.from_numpy(rows).to(DEV)], pos[:, rows], axes, exact,
               inter, m, inverse)
    # the farthest positions: the same angles from reduced ones
    turns = np.array([[int(pos[a, 0]) * int(s) % 2 ** 64 for s in steps] for a in range(n)], dtype=object)
    angle = np.array([float(turns[a][i]) / 2.0 ** 64 * 2 * np.pi for i, a in enumerate(axes)])
    _check(qo[:1], q[:1], np.ones((n, 1)), axes, angle, inter, m, inverse)


def test_one_axis_is_the_plain_call(lib):
    """Positions of one axis that go on as the documents do: the same bits, also with
    the same positions on three axes."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(3)
    n, starts, d = [5, 0, 600, 1], [7, 3, 0, 131071], 128
    T = sum(n)
    w = fl.rope_frequencies(d, factor=4.0, method="bands")
    q, k = bf16(rng, (T, 4, d)).to(DEV), bf16(rng, (T, 2, d)).to(DEV)
    want = fl.Rotary(w)(q, k, offsets(n), i32(starts))
    pos = i32(np.concatenate([np.arange(s, s + c) for s, c in zip(starts, n)]))[None]
    for axes, p in (([0] * 64, pos), (fl.rope_axes([16, 24, 24]), pos.expand(3, T)),
                    (fl.rope_axes([22, 21, 21], cyclic=True), pos.repeat(4, 1))):
        got = fl.Rotary(w, axes=axes)(q, k, offsets(n), positions=p)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_padding_strides_and_in_place(lib):
    """Rows behind the last document stay as they were; rows of a packed projection,
    turned in place; a slice of a longer table of positions."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(4)
    for T, end in ((9, 5), (900, 777), (8, 0)):
        H, H_kv, d = 4, 2, 64
        x = bf16(rng, (T, (H + 2 * H_kv) * d)).to(DEV)
        keep = x.clone()
        q, k = x[:, :H * d].view(T, H, d), x[:, H * d:(H + H_kv) * d].view(T, H_kv, d)
        q0, k0 = q.clone(), k.clone()
        pos = torch.from_numpy(rng.integers(0, 5000, (3, T + 11)).astype(np.int32)).to(DEV)
        rope = fl.Rotary(fl.rope_frequencies(d), axes=fl.rope_axes([8, 12, 12]))
        rope(q, k, offsets([end // 2, end - end // 2]), positions=pos[:, 4:4 + T], q_out=q, k_out=k)
        assert torch.equal(x[end:], keep[end:]) and torch.equal(x[:, (H + H_kv) * d:], keep[:, (H + H_kv) * d:])
        if end:
            p = pos[:, 4:4 + end].cpu().numpy()
            w = fl.rope_frequencies(d).numpy()
            _check(q[:end], q0[:end], p, fl.rope_axes([8, 12, 12]), w, False, 1.0, False)
            _check(k[:end], k0[:end], p, fl.rope_axes([8, 12, 12]), w, False, 1.0, False)


def test_the_inverse_is_the_gradient(lib):
    """<R x, y> = <x, R^T y>: the gradient of a sum over turned rows, against differences
    of the (linear) forward; within the outputs' BF16 roundings."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(6)
    T, H, d = 64, 2, 64
    rope = fl.Rotary(fl.rope_frequencies(48), interleaved=True, mscale=1.5, axes=fl.rope_axes([9, 8, 7], cyclic=True))
    pos = torch.from_numpy(rng.integers(0, 300, (3, T)).astype(np.int32)).to(DEV)
    cu = offsets([T])
    g = bf16(rng, (T, H, d)).to(DEV)
    dx, _ = rope(g, None, cu, positions=pos, inverse=True)
    zero = torch.zeros(T, H, d, dtype=torch.bfloat16, device=DEV)
    for e in (0, 1, 7, 46, 47, 48, 63):
        x = zero.clone()
        x[:, :, e] = 1
        y, _ = rope(x, None, cu, positions=pos)
        slope = (y.double() * g.double()).sum(2)
        size = (y.double().abs() * g.double().abs()).sum(2)
        assert ((slope - dx[:, :, e].double()).abs() <= 2 * TOL * size + 2.0 ** -100).all()
