"""What the Python binding hands to the cached attention (no GPU: the library's entry
point is replaced, and CPU tensors count as being on the current device)."""
import types

import numpy as np
import pytest
import torch


@pytest.fixture
def attend(monkeypatch):
    from precision_causal_attention_block_gb300 import flamia as fl
    calls = []

    class Lib:
        def flamia_attn_cache(self, *a):
            calls.append(a)
            return 0

    monkeypatch.setattr(fl, "_LIB", Lib())
    monkeypatch.setattr(fl, "_current", lambda: (-1, 0))
    cache = types.SimpleNamespace(d=64, H_kv=2, device_index=-1, _ref=None)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    big = torch.zeros(4096, dtype=torch.uint8)

    def run(scale=0.125, window=0, sinks=0, ws=big):
        fl.flamia_attn_cache(cache, q, cu, None, table, scale, window, sinks, torch.empty_like(q),
                             None, ws)
        return calls[-1]

    run.calls = calls
    run.big = big
    return run


def test_a_workspace_is_one_piece_of_memory(attend):
    """An expanded tensor has as many bytes as its shape says and owns one of them."""
    a = attend()
    assert a[15] == attend.big.data_ptr() and a[16] == 4096
    n = len(attend.calls)
    for ws in (attend.big[:1].expand(1 << 26), attend.big[::2], attend.big.view(64, 64).t()):
        with pytest.raises(RuntimeError, match="ws"):
            attend(ws=ws)
    assert len(attend.calls) == n


def test_windows_and_first_tokens_beyond_32_bits(attend):
    """They see the same as the largest of 32 bits; negative ones stay negative."""
    top = (1 << 31) - 1
    for given, want in ((0, 0), (5, 5), (top, top), (top + 1, top), ((1 << 32) + 5, top),
                        (1 << 63, top), (-1, -1), (-(1 << 32), -1), (5 - (1 << 32), -1)):
        a = attend(window=given, sinks=0)
        assert (a[11], a[12]) == (want, 0), given
        a = attend(window=7, sinks=given)
        assert (a[11], a[12]) == (7, want), given


def test_any_number_is_a_scale(attend):
    for s in (0.25, 1, np.float32(0.25), np.float64(0.25), torch.tensor(0.25)):
        assert type(attend(scale=s)[10]) is float


def test_arguments_by_position_keep_their_places():
    """What a training call took by position before it knew rotary positions."""
    import inspect
    from precision_causal_attention_block_gb300 import flamia as fl
    names = list(inspect.signature(fl.TrainingCall).parameters)
    assert names[:17] == ["T", "H", "d", "cu_seqlens", "softmax_scale", "nvfp4_qk", "hadamard", "causal",
                          "H_kv", "deterministic_dq", "dq_accum", "schedule", "ds_rows", "token_scales",
                          "ds_zero_count", "bwd_ctas", "device"]


def test_turns_are_rounded():
    """round(2^64 w / 2 pi), as the C header has it, for slow pairs too."""
    from fractions import Fraction
    from precision_causal_attention_block_gb300 import flamia as fl
    import math
    w = [1e-9, 3e-12, 7.7e-15, 0.01]
    r = fl.Rotary(w, device="cpu")
    for f, t in zip(w, r.turns.tolist()):
        x = Fraction(f / (2 * math.pi)) * 2 ** 64
        assert abs(t - x) <= Fraction(1, 2), f
