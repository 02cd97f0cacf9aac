"""The rotary and cache oracle against closed forms, differences and the
training quantiser's oracle."""
import numpy as np
import pytest

from oracle import flamia_oracle as O
from oracle import serving_oracle as S


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_and_inverse_its_transpose(interleaved):
    rng = np.random.default_rng(0)
    x, g = rng.standard_normal((2, 5, 3, 64))
    pos, w = np.array([0, 1, 7, 1000, 131071]), 10000.0 ** (-np.arange(0, 48, 2) / 48)
    y = S.rope(x, pos, w, interleaved, 1.25)
    # relative positions: <R(p) a, R(q) b> depends on p - q alone
    a = S.rope(x[:1], [10], w, interleaved), S.rope(g[:1], [4], w, interleaved)
    b = S.rope(x[:1], [1006], w, interleaved), S.rope(g[:1], [1000], w, interleaved)
    assert np.allclose((a[0] * a[1]).sum(-1), (b[0] * b[1]).sum(-1), atol=1e-9)
    assert np.array_equal(y[..., 48:], x[..., 48:]) and np.array_equal(y[0, :, :48], 1.25 * x[0, :, :48])
    back = S.rope(g, pos, w, interleaved, 1.25, inverse=True)
    assert np.allclose((y * g).sum(), (x * back).sum())
    # and against differences of the scalar <y, g>
    eps = 1e-5
    for i in ((1, 0, 3), (3, 2, 40), (4, 1, 60)):
        z = x.copy()
        z[i] += eps
        d = ((S.rope(z, pos, w, interleaved, 1.25) * g).sum() - (y * g).sum()) / eps
        assert abs(d - back[i]) < 1e-4


@pytest.mark.parametrize("token", [False, True])
def test_prompt_write_is_the_training_quantiser(token):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((77, 2, 64)) * rng.uniform(0.1, 30, (77, 1, 1))
    codes, sb = O.quantize_tokenblock(x, [0, 77], group="token" if token else "block")
    c = S.Cache(1, 2, 64, token)
    c.write(0, x, 0)
    assert np.array_equal(c.codes[0], codes) and np.array_equal(c.scales[0], sb.T)


def test_growing_block_rounds_held_codes_again():
    c = S.Cache(1, 1, 64)
    one = np.full((1, 1, 64), 3.3)
    c.write(0, one, 0)
    first = c.values(0)[0, 0, 0]
    c.write(0, one * 100, 1)
    assert c.scales[0][0, 0] == c.scales[0][1, 0]
    assert abs(c.values(0)[0, 0, 0] - first) <= 2.0 ** (int(c.scales[0][1, 0]) - 127) * 3.3 * 2.0 ** -4
    before = c.codes[0].copy()
    c.write(0, one * 100, 1)  # the same call again changes nothing
    assert np.array_equal(before, c.codes[0])
    c.write(0, one / 100, 2)  # a small token keeps the block's exponent
    assert c.scales[0][2, 0] == c.scales[0][1, 0] and np.array_equal(before[:2], c.codes[0][:2])


def test_seen_keys():
    assert S.seen_keys(4, 10).tolist() == [True] * 5 + [False] * 5
    assert S.seen_keys(-1, 3).sum() == 0
    assert np.nonzero(S.seen_keys(9, 12, window=3))[0].tolist() == [7, 8, 9]
    assert np.nonzero(S.seen_keys(9, 12, window=3, sinks=2))[0].tolist() == [0, 1, 7, 8, 9]
    assert np.nonzero(S.seen_keys(1, 12, window=3, sinks=4))[0].tolist() == [0, 1]
    assert np.nonzero(S.seen_keys(5, 6, window=6, sinks=4))[0].tolist() == [0, 1, 2, 3, 4, 5]


def test_attend_of_one_key_is_its_value():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 2, 64))
    o, lse = S.attend(q, k, v, 0, 0.125, window=1)
    assert np.allclose(o, v) and np.allclose(lse.T, 0.125 * (q * k).sum(-1))
    full, l2 = S.attend(q, k, v, 0, 0.125)
    ref = O.attention(q, k, v, np.zeros_like(q), [0, 4], 0.125, quant=False)
    assert np.allclose(full, ref["O"])


def test_rope_frequencies():
    from precision_causal_attention_block_gb300 import flamia as fl
    w = fl.rope_frequencies(64).numpy()
    assert np.allclose(w, 10000.0 ** (-np.arange(0, 64, 2) / 64)) and w[0] == 1.0
    assert np.allclose(fl.rope_frequencies(64, factor=4.0).numpy(), w / 4)
    b = fl.rope_frequencies(64, factor=4.0, method="base").numpy()
    assert b[0] == 1.0 and np.isclose(b[-1], w[-1] / 4)
    m = fl.rope_frequencies(64, factor=4.0, method="bands", original_len=4096).numpy()
    turns = 4096 * w / (2 * np.pi)
    assert np.array_equal(m[turns >= 4], w[turns >= 4])
    assert np.allclose(m[turns <= 1], w[turns <= 1] / 4)
    assert np.all(m <= w) and np.all(m >= w / 4)
    for bad in (dict(rot_dim=15), dict(rot_dim=64, method="other")):
        with pytest.raises(ValueError):
            fl.rope_frequencies(**bad)
    # the table of turns: round(2^64 w / 2 pi), exact for a quarter turn
    r = fl.Rotary([np.pi / 2, np.pi, 1e-3], device="cpu")
    assert r.turns.tolist()[:2] == [1 << 62, -(1 << 63)] and r.rot_dim == 6
    assert abs(r.turns.tolist()[2] - 1e-3 / (2 * np.pi) * 2.0 ** 64) <= 2.0 ** 12
