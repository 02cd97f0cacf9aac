"""The paged cache on the GPU: codes and scale bytes bit for bit the oracle's,
read back exactly."""
import numpy as np
import pytest
import torch

from tests.serving_helpers import DEV, Pair, bf16, i32, offsets, page_table

pytestmark = pytest.mark.gpu


def _steps(rng, nseq, steps):
    """Token counts of several calls: prompts, single tokens, idle sequences."""
    out = []
    for i in range(steps):
        n = rng.integers(0, 70, nseq) if i % 3 == 0 else rng.integers(0, 2, nseq)
        if n.sum() == 0:
            n[0] = 1
        out.append([int(x) for x in n])
    return out


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("d,H_kv,page", [(64, 1, 32), (64, 3, 64), (128, 2, 128), (128, 5, 32),
                                         (128, 1, 384)])
def test_writes_in_pieces(lib, d, H_kv, page, token):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(d + H_kv + page)
    nseq = 5
    steps = _steps(rng, nseq, 7)
    lens = np.zeros(nseq, dtype=int)
    pair = Pair(fl, rng, np.sum(steps, axis=0), page, H_kv, d, token)
    for n in steps:
        T = sum(n)
        # growing magnitudes, so that held blocks are rounded again
        k = bf16(rng, (T, H_kv, d)) * float(2.0 ** rng.integers(-3, 6))
        v = bf16(rng, (T, H_kv, d)) * float(2.0 ** rng.integers(-3, 6))
        pair.write(k, v, n, [int(s) for s in lens])
        lens += n
        pair.check_equal(lens)
    # positions behind the last token keep what they held
    got = pair.gpu.k_codes.cpu().numpy()
    for b in range(nseq):
        p = np.arange(lens[b], -(-lens[b] // page) * page)
        assert (got[pair.t[b, p // page], :, p % page] == 0x7F).all()
    assert int(pair.status.item()) == 0
    # and the read-back is exact: every cached value is a BF16 number here
    n = [int(x) for x in lens]
    k, v = pair.gpu.read(offsets(n), i32([0] * nseq), pair.table, sum(n))
    assert np.array_equal(k.double().cpu().numpy(), np.concatenate([pair.k.values(b) for b in range(nseq)]))
    assert np.array_equal(v.double().cpu().numpy(), np.concatenate([pair.v.values(b) for b in range(nseq)]))
    # a part of each sequence, from odd positions on
    part, start = [x // 2 for x in n], [x // 3 for x in n]
    k, _ = pair.gpu.read(offsets(part), i32(start), pair.table, sum(part))
    want = np.concatenate([pair.k.values(b)[start[b]:start[b] + part[b]] for b in range(nseq)])
    assert np.array_equal(k.double().cpu().numpy(), want)


@pytest.mark.parametrize("token", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_gets_the_training_quantisers_codes(lib, d, token):
    """A prompt written at position 0 holds the codes and scales of
    flamia_quantize_tokenblock bit for bit."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(d)
    n, H = [130, 1, 64, 33], 3
    T = sum(n)
    x = (bf16(rng, (T, H, d)) * torch.from_numpy(2.0 ** rng.integers(-140, 120, (T, 1, 1)))).to(torch.bfloat16)
    x[5] = 0
    x[131:163] = 0
    xd = x.to(DEV)
    cu = offsets(n)
    ref = fl.QTensor(T, H, d)
    fl.flamia_quantize_tokenblock(xd, cu, ref, fl.FORMAT_TOKEN_SCALES if token else fl.FORMAT_MXFP8)
    t, pages = page_table(rng, n, 64)
    c = fl.KVCache(pages, 64, H, d, token_scales=token)
    c.write(xd, xd, cu, None, torch.from_numpy(t).to(DEV))
    at = 0
    for b, m in enumerate(n):
        p = torch.arange(m, device=DEV)
        pg = torch.from_numpy(t).to(DEV).long()[b, p // 64]
        for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
            assert torch.equal(codes[pg, :, p % 64], ref.codes[at:at + m])
            assert torch.equal(scales[pg, :, p % 64], ref.scales[:, at:at + m].t())
        at += m


def test_extreme_values(lib):
    """Largest and smallest BF16 numbers, zeros, infinities and NaN: bit for bit the
    oracle's codes; NaN codes where the input was not finite, the others unmoved."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(9)
    n = [40, 40, 40]
    x = bf16(rng, (120, 2, 64))
    x[0, 0, 0] = 3.3e38
    x[41, 1, 5] = float("inf")
    x[45, 1, 6] = float("-inf")
    x[42, 0, 7] = float("nan")
    x[80:, 0] = 0
    x[80:, 1] = 1e-39
    pair = Pair(fl, rng, [n_ + 1 for n_ in n], 64, 2, 64)
    pair.write(x, -x, n, [0, 0, 0])
    pair.check_equal(n)
    # a block that holds NaN codes is rounded again around them
    y = torch.full((3, 2, 64), 1000.0, dtype=torch.bfloat16)
    pair.write(y, y, [1, 1, 1], n)
    pair.check_equal([41, 41, 41])
    assert int(pair.status.item()) == 0


def test_repeated_write_changes_nothing_and_strided_rows(lib):
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(11)
    n, starts, H, d = [1, 3, 40], [31, 30, 95], 2, 128
    pair = Pair(fl, rng, [s + m for s, m in zip(starts, n)], 32, H, d)
    first = bf16(rng, (sum(starts), H, d))
    pair.write(first, first, starts, [0, 0, 0])
    x = bf16(rng, (sum(n), 3 * H, d), 8.0).to(DEV)
    k, v = x[:, H:2 * H], x[:, 2 * H:]  # slices of a packed projection
    assert not k.is_contiguous()
    pair.gpu.write(k, v, offsets(n), i32(starts), pair.table)
    one = [t.clone() for t in (pair.gpu.k_codes, pair.gpu.k_scales, pair.gpu.v_codes)]
    pair.gpu.write(k, v, offsets(n), i32(starts), pair.table)
    assert all(torch.equal(a, b) for a, b in zip(one, (pair.gpu.k_codes, pair.gpu.k_scales,
                                                       pair.gpu.v_codes)))
    at = 0
    for b, m in enumerate(n):
        pair.k.write(b, k[at:at + m].double().cpu().numpy(), starts[b])
        pair.v.write(b, v[at:at + m].double().cpu().numpy(), starts[b])
        at += m
    pair.check_equal([s + m for s, m in zip(starts, n)])


def test_padded_batch_and_bad_pages(lib):
    """Rows behind the last sequence are neither written nor read; a bad page, a
    position outside the table and a negative start are reported, and the other
    sequences are served."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(12)
    H, d, page = 1, 64, 32
    c = fl.KVCache(6, page, H, d)
    x = bf16(rng, (8, H, d)).to(DEV)
    for table, starts, cu in (([[0], [6]], [0, 0], [0, 2, 4]), ([[0], [-1]], [0, 0], [0, 2, 4]),
                              ([[0], [1]], [0, 32], [0, 2, 4]), ([[0], [1]], [0, -1], [0, 2, 4]),
                              ([[0], [1 << 30]], [0, 0], [0, 2, 4]),
                              ([[0], [1]], [0, (1 << 31) - 3], [0, 2, 4])):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        c.k_codes.zero_()
        c.write(x, x, i32(cu), i32(starts), torch.tensor(table, dtype=torch.int32, device=DEV),
                dev_status=st)
        assert int(st.item()) == fl.DEV_BAD_PAGE, (table, starts)
        assert bool(c.k_codes[0, 0, :2].any()) and not bool(c.k_codes[1:].any())
        assert not bool(c.k_codes[0, 0, 2:].any())
        out = torch.full((8, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
        st.zero_()
        c.read(i32(cu), i32(starts), torch.tensor(table, dtype=torch.int32, device=DEV), 8,
               k_out=out, v_out=out.clone(), dev_status=st)
        assert int(st.item()) == fl.DEV_BAD_PAGE
        assert bool((out[2:] == 7.0).all()) and not bool((out[:2] == 7.0).all())
    # malformed offsets
    for cu in ([0, 9], [0, 5, 3], [2, 8]):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        n = len(cu) - 1
        c.write(x, x, i32(cu), i32([0] * n), torch.zeros(n, 1, dtype=torch.int32, device=DEV),
                dev_status=st)
        assert int(st.item()) & fl.DEV_BAD_SEQLENS


def test_many_single_tokens(lib):
    """700 sequences, one token each, at every offset of a block."""
    from precision_causal_attention_block_gb300 import flamia as fl
    rng = np.random.default_rng(13)
    nseq, H, d = 700, 2, 64
    starts = [i % 67 for i in range(nseq)]
    pair = Pair(fl, rng, [s + 1 for s in starts], 64, H, d)
    x = bf16(rng, (sum(starts), H, d))
    pair.write(x, x, starts, [0] * nseq)
    y = bf16(rng, (nseq, H, d), 2.0)
    pair.write(y, y, [1] * nseq, starts)
    pair.check_equal([s + 1 for s in starts])
    assert int(pair.status.item()) == 0
