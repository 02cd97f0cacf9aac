"""Windows, first tokens and half-seen NaN in the kernels of 8 and 16 query rows an
item (single and drafted tokens), over contexts of many key tiles."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, Pair, bf16, check_attend, i32, offsets
from tests.test_gpu_attn_cache import _run, test_many_tiles_a_cta as many_tiles

pytestmark = pytest.mark.gpu


def _rows(n, H, H_kv, want):
    """Rows an item: the kernel's rule on the mean of a sequence and K / V head."""
    rows = -(-sum(n) // len(n)) * (H // H_kv)
    assert (8 if rows <= 8 else 16 if rows <= 16 else 32 if rows <= 96 else 256) == want, rows


WINDOWS = [(1, 0), (1, 1), (7, 4), (32, 0), (100, 130), (128, 4), (129, 64), (300, 1), (900, 260),
           (5000, 3)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("token", [False, True])
def test_window_and_first_tokens(lib, window, sinks, token):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(window + sinks)
    for n, starts, H, H_kv, d, page, want in (
            ([1, 1, 1, 1, 1], [700, 383, 0, 2500, 128], 4, 2, 64, 32, 8),
            ([1, 1], [3000, 90], 8, 1, 128, 128, 8),
            ([2, 1, 2], [1500, 255, 130], 8, 2, 128, 64, 8),
            ([4, 2, 4], [1700, 511, 0], 4, 1, 64, 64, 16),
            ([3, 4], [257, 2100], 16, 4, 128, 32, 16),
            ([13], [1151], 1, 1, 64, 256, 16)):
        _rows(n, H, H_kv, want)
        _run(fl, rng, n, starts, H, H_kv, d, page, token, window=window, sinks=sinks)


LONG_RUNS = [
    # sequences, longest context, new tokens, H, H_kv, d, page, window, sinks
    (120, 2500, 1, 16, 8, 128, 64, 700, 4),
    (120, 2500, 1, 16, 16, 64, 32, 300, 130),
    (40, 6000, 1, 32, 4, 128, 128, 2000, 260),
    (90, 2500, 4, 16, 8, 128, 64, 500, 130),
]


@pytest.mark.parametrize("nseq,longest,new,H,H_kv,d,page,window,sinks", LONG_RUNS)
def test_many_tiles_a_cta(lib, nseq, longest, new, H, H_kv, d, page, window, sinks):
    many_tiles(lib, nseq, longest, new, H, H_kv, d, page, window, sinks)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("n,H,d,want", [(1, 4, 64, 8), (1, 16, 128, 8), (4, 4, 128, 8),
                                        (6, 4, 64, 16), (8, 4, 128, 16)])
def test_nan_stays_where_it_is_seen(lib, n, H, d, want, which):
    """As for many rows: NaN keys and values outside the window, behind the end or in
    another sequence change nothing; of a sequence's drafts those that see one are NaN."""
    from precision_causal_attention_block_gb300 import flamia as fl
    L, H_kv, window = 700, 2, 150
    _rows([n, n, n], H, H_kv, want)
    outs = []
    for plant in (True, False):
        rng = np.random.default_rng(61)
        pair = Pair(fl, rng, [L, L, L], 32, H_kv, d, True)  # (exponents of single tokens)
        k, v = (bf16(rng, (3 * L, H_kv, d)) for _ in range(2))
        q = bf16(rng, (3 * n, H, d)).to(DEV)
        if plant:
            x = k if which == "k" else v
            x[100, :, 3] = float("nan")                       # sequence 0: behind every window
            x[L + L - n // 2 - 1, 0, 5] = float("inf")        # 1: the later drafts see it
            x[2 * L + L - n - window + 1, 1, 0] = float("nan")  # 2: the first draft's last key
        pair.write(k, v, [L] * 3, [0] * 3)
        args = offsets([n] * 3), i32([L - n] * 3), pair.table, d ** -0.5
        outs.append(pair.gpu.attend(q, *args, window=window)[0])
        if not plant:
            o, lse = pair.gpu.attend(q, *args, window=window)
            check_attend(o, lse, pair, q, [n] * 3, [L - n] * 3, d ** -0.5, window)
    G = H // H_kv
    bad = np.zeros((3 * n, H), dtype=bool)
    bad[n + n - n // 2 - 1:2 * n, :G] = True
    bad[2 * n, G:] = True
    nan = torch.isnan(outs[0]).cpu().numpy()
    assert np.array_equal(nan.any(-1), bad)
    got, ref = outs[0].cpu(), outs[1].cpu()
    keep = torch.from_numpy(~bad)
    assert torch.equal(got[keep], ref[keep])
