"""Positions that a call has no use for, or lacks, are refused before anything is done."""
import types

import pytest
import torch


def _ropes(fl):
    w = fl.rope_frequencies(16)
    return fl.Rotary(w, device="cpu"), fl.Rotary(w, device="cpu", axes=[0] * 4 + [1] * 4)


def test_training_call():
    from precision_causal_attention_block_gb300 import flamia as fl
    plain, axes = _ropes(fl)
    pos = torch.zeros(2, 3, dtype=torch.int32)
    for rope, positions in ((None, pos), (plain, pos), (axes, None)):
        call = fl.TrainingCall.__new__(fl.TrainingCall)  # (its buffers need a GPU)
        call.rope = rope
        for run in (lambda: call.forward(None, None, None, positions=positions),
                    lambda: call(None, None, None, None, positions=positions)):
            with pytest.raises(RuntimeError, match="positions"):
                run()


def test_decode_call_leaves_the_books():
    from precision_causal_attention_block_gb300 import flamia as fl
    plain, axes = _ropes(fl)
    pos = torch.zeros(2, 3, dtype=torch.int32)
    did = []
    cache = types.SimpleNamespace(write=lambda *a, **k: did.append("write"),
                                  attend=lambda *a, **k: did.append("attend"))
    pool = types.SimpleNamespace(reserve=lambda *a, **k: did.append("reserve"), page_table=None)
    for rope, positions in ((None, pos), (plain, pos), (axes, None)):
        call = fl.DecodeCall.__new__(fl.DecodeCall)
        vars(call).update(cache=cache, pool=pool, rope=rope, T=3, granted=None, status=None)
        with pytest.raises(RuntimeError, match="positions"):
            call(None, None, None, None, None, positions=positions)
    assert did == []
