"""Cached tokens written again while later ones of their block stay: the rows of a
block then have exponents of their own, and each keeps its value."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, Pair, bf16, i32, offsets

pytestmark = pytest.mark.gpu


def _values(pair, b, n):
    k, v = pair.gpu.read(offsets([n]), i32([0]), pair.table[b:b + 1].contiguous(), n)
    return k.double().cpu().numpy(), v.double().cpu().numpy()


@pytest.mark.parametrize("d,H_kv,page", [(64, 2, 32), (128, 3, 64)])
@pytest.mark.parametrize("again", [0, 3])
@pytest.mark.parametrize("last", [0.25, 4.0, 2.0 ** 9])
def test_a_part_written_again_under_a_smaller_exponent(lib, d, H_kv, page, again, last):
    """Ten small tokens, five large ones, a part of the small ones once more, then a
    token of any size behind them: the large ones keep their values to the half
    steps of at most three roundings (when written, and when the block's exponent grows)."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(d + again)
    pair = Pair(fl, rng, [64], page, H_kv, d)
    x = bf16(rng, (16, H_kv, d))
    x[10:15] *= 64.0
    x[15] *= last
    lens = 0
    for a, e in ((0, 10), (10, 15), (again, 10), (15, 16)):
        pair.write(x[a:e], -x[a:e], [e - a], [a])
        lens = max(lens, e)
        pair.check_equal([lens])
    k, v = _values(pair, 0, 16)
    want = x.double().numpy()
    step = 2.0 ** np.ceil(np.log2(np.abs(want).max(axis=(0, 2)) / 448))[None, :, None]
    # E4M3: half a step is 2^-4 of the value (of the third rounding's operand: 1.13 times
    # it), or 2^-10 of the scale below its normal range
    tol = 3 * 1.13 * (2.0 ** -4 * np.abs(want) + 2.0 ** -10 * step)
    assert (np.abs(k - want) <= tol).all() and (np.abs(v + want) <= tol).all()
    assert int(pair.status.item()) == 0


def test_random_rewrites(lib):
    """Any order of writes that start inside what a sequence holds: codes and scale
    bytes bit for bit the oracle's, tokens behind a write as they were."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(71)
    nseq, H_kv, d = 9, 2, 64
    pair = Pair(fl, rng, [160] * nseq, 32, H_kv, d)
    lens = [0] * nseq
    for _ in range(25):
        starts = [int(rng.integers(0, c + 1)) for c in lens]
        n = [int(min(160 - s, rng.integers(0, 50))) for s in starts]
        n[0] = max(n[0], 1) if starts[0] < 160 else 0
        if sum(n) == 0:
            continue
        k, v = (bf16(rng, (sum(n), H_kv, d)) * float(2.0 ** rng.integers(-4, 5)) for _ in range(2))
        pair.write(k, v, n, starts)
        lens = [max(c, s + m) for c, s, m in zip(lens, starts, n)]
        pair.check_equal(lens)
    assert int(pair.status.item()) == 0
