"""Workloads of the serving and rotary operators: what is timed, and what each
result is compared with.

Five operators around the packed MXFP8 attention:

* ``rope`` / ``rope_bwd``: rotary positions of Q and K (and of dQ and dK);
* ``write`` / ``read``: the paged key-value cache in E4M3 codes with one E8M0
  exponent per 32-token block and head (or per token and head);
* ``attend``: attention of new tokens over that cache, optionally over a
  sliding window and the first tokens only.

``run`` computes them from elementary torch operations (``own`` false) or
through the library's entry points (``own`` true) on the same state.
"""
import json
import math
import zlib

import torch

own = False

DEV = "cuda"
BLOCK = 32


# ------------------------------------------------------------------ cases

def listed():
    """Twelve cases; the head shapes are those of the training workloads (16
    heads of 128, 32 heads of 64) and grouped-query forms of them."""
    return [
        # one decode step of 16 sequences: latency
        {"name": "rope_decode", "op": "rope", "batch": 16, "lo": 1, "hi": 1, "H": 32, "H_kv": 8, "d": 128,
         "rot": 128, "interleaved": False, "factor": 1.0, "ctx": 131072},
        # the long-context training call's Q and K before quantisation
        {"name": "rope_long", "op": "rope", "batch": 1, "lo": 131072, "hi": 131072, "H": 32, "H_kv": 32, "d": 64,
         "rot": 64, "interleaved": False, "factor": 8.0, "ctx": 0},
        # dQ and dK of the 4 x 4096 training call, half of each head rotated
        {"name": "rope_bwd_packed", "op": "rope_bwd", "batch": 4, "lo": 4096, "hi": 4096, "H": 16, "H_kv": 16, "d": 128,
         "rot": 64, "interleaved": True, "factor": 1.0, "ctx": 0},
        # one decode step of 64 sequences written behind what they hold
        {"name": "write_decode", "op": "write", "batch": 64, "lo": 1, "hi": 1, "H_kv": 8, "d": 128, "page": 64,
         "ctx": 4096, "token_scales": False},
        # prompts of very different length into an empty cache
        {"name": "write_prompts", "op": "write", "batch": 40, "lo": 1, "hi": 16384, "H_kv": 16, "d": 128, "page": 128,
         "ctx": 0, "token_scales": False},
        # short contexts brought back as BF16
        {"name": "read_short", "op": "read", "batch": 4, "lo": 33, "hi": 517, "H_kv": 4, "d": 64, "page": 32, "ctx": 96},
        # long contexts brought back as BF16
        {"name": "read_long", "op": "read", "batch": 8, "lo": 5000, "hi": 16384, "H_kv": 16, "d": 128, "page": 128, "ctx": 1024},
        # one short conversation, one token: latency
        {"name": "attend_one", "op": "attend", "batch": 1, "new_lo": 1, "new_hi": 1, "ctx_lo": 257, "ctx_hi": 257,
         "H": 16, "H_kv": 16, "d": 128, "page": 64, "window": 0, "sinks": 0},
        # a serving batch with contexts of very different length, grouped heads
        {"name": "attend_batch", "op": "attend", "batch": 96, "new_lo": 1, "new_hi": 1, "ctx_lo": 16, "ctx_hi": 16384,
         "H": 32, "H_kv": 8, "d": 128, "page": 64, "window": 0, "sinks": 0},
        # one token over the longest training context
        {"name": "attend_long", "op": "attend", "batch": 1, "new_lo": 1, "new_hi": 1, "ctx_lo": 131072, "ctx_hi": 131072,
         "H": 32, "H_kv": 32, "d": 64, "page": 256, "window": 0, "sinks": 0},
        # four drafted tokens a sequence, a window and four first tokens
        {"name": "attend_window", "op": "attend", "batch": 48, "new_lo": 4, "new_hi": 4, "ctx_lo": 2000, "ctx_hi": 20000,
         "H": 16, "H_kv": 4, "d": 128, "page": 32, "window": 4096, "sinks": 4},
        # the next chunk of a long prompt over what is cached
        {"name": "attend_chunk", "op": "attend", "batch": 2, "new_lo": 500, "new_hi": 512, "ctx_lo": 7000, "ctx_hi": 8192,
         "H": 16, "H_kv": 16, "d": 128, "page": 128, "window": 0, "sinks": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "write", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128])
    H_kv = rng.choice([1, 2, 4, 5, 8, 16])
    H = H_kv * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * H_kv <= 32])
    batch = _log(rng, 1, 96)
    page = rng.choice([32, 64, 128, 256])
    if op in ("rope", "rope_bwd"):
        tokens = _log(rng, 1, 65536)
        n = max(1, tokens // batch)
        return {"op": op, "batch": batch, "lo": max(1, n // 2), "hi": n, "H": H, "H_kv": H_kv, "d": d,
                "rot": rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d]),
                "interleaved": rng.random() < 0.5, "factor": rng.choice([1.0, 4.0, 8.0]),
                "ctx": rng.choice([0, _log(rng, 1, 131072)])}
    if op in ("write", "read"):
        tokens = _log(rng, 1, 65536)
        n = max(1, tokens // batch)
        c = {"op": op, "batch": batch, "lo": max(1, n // 2), "hi": n, "H_kv": H_kv, "d": d, "page": page,
             "ctx": rng.choice([0, _log(rng, 1, 4096)])}
        if op == "write":
            c["token_scales"] = rng.random() < 0.3
        return c
    new = rng.choice([1, 1, 1, _log(rng, 1, 8), _log(rng, 1, 256)])
    total = min(_log(rng, 256, 600000), int(3e9 / (new * H * d)), int(2.5e8 / (H_kv * d)))
    hi = max(new, total // batch, 16)
    windowed = rng.random() < 0.4
    return {"op": "attend", "batch": batch, "new_lo": max(1, new // 2), "new_hi": new, "ctx_lo": max(new, hi // 3),
            "ctx_hi": hi, "H": H, "H_kv": H_kv, "d": d, "page": page, "window": _log(rng, 1, hi) if windowed else 0,
            "sinks": rng.choice([0, 1, 4, 64]) if windowed else 0}


# ------------------------------------------------------------------ inputs

def _between(gen, n, lo, hi):
    """n whole numbers in [lo, hi], spread over their logarithm where that is wide."""
    u = torch.rand(n, generator=gen, dtype=torch.float64)
    if hi > 10 * lo:
        x = torch.exp(math.log(max(lo, 1)) + u * (math.log(hi) - math.log(max(lo, 1)))).round()
    else:
        x = lo + (u * (hi - lo + 1)).floor()
    return x.clamp(lo, hi).to(torch.int64)


def _lengths(case):
    """(new tokens, tokens cached before them) of every sequence: a case's own,
    whatever the seed."""
    c = case
    gen = torch.Generator().manual_seed(zlib.crc32(json.dumps(
        {k: v for k, v in c.items() if k != "name"}, sort_keys=True).encode()))
    if c["op"] == "attend":
        n = _between(gen, c["batch"], c["new_lo"], c["new_hi"])
        return n, torch.maximum(_between(gen, c["batch"], c["ctx_lo"], c["ctx_hi"]), n) - n
    n = _between(gen, c["batch"], c["lo"], c["hi"])
    return n, _between(gen, c["batch"], 0, c["ctx"]) if c["ctx"] else torch.zeros_like(n)


def _offsets(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])


def _int32(x):
    return x.to(torch.int32).to(DEV)


def _normal(gen, shape, rms=None):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    if rms is not None:
        x *= rms
    return x.to(torch.bfloat16)


def _head_rms(gen, H):
    """Per-head RMS in [0.5, 2], as in the training workloads."""
    return 0.5 + 1.5 * torch.rand(H, generator=gen, device=DEV)[:, None]


def _pow2(byte):
    """2^(byte - 127) as float32, from E8M0 bytes."""
    b = byte.to(torch.int32)
    return torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)


def _scale_byte(amax):
    """E8M0 byte of the smallest e with amax <= 448 * 2^e, e in [-127, 127]."""
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    return (e.clamp(-127, 127) + 127).to(torch.int32)


def _codes(x, byte):
    """E4M3 codes of x * 2^-(byte - 127)."""
    return (x * _pow2(254 - byte)).to(torch.float8_e4m3fn)


def _table(gen, lens, page):
    """Page table of sequences of these lengths: the pages in random order, -1
    where a sequence needs none."""
    need = (lens + page - 1) // page
    width = max(1, int(need.max()))
    pages = int(need.sum())
    order = torch.randperm(max(pages, 1), generator=gen)
    table = torch.full((lens.numel(), width), -1, dtype=torch.int64)
    first = _offsets(need)
    for b in range(lens.numel()):
        n = int(need[b])
        table[b, :n] = order[int(first[b]):int(first[b]) + n]
    return _int32(table), max(pages, 1)


def _filled(gen, pages, H_kv, page, d):
    """A pool of pages as a block-scaled write leaves it: codes and scale bytes."""
    x = _normal(gen, (pages, H_kv, page, d), _head_rms(gen, H_kv)[None, :, :, None]).float()
    x = x.view(pages, H_kv, page // BLOCK, BLOCK, d)
    byte = _scale_byte(x.abs().amax((3, 4), keepdim=True))
    codes = _codes(x, byte).view(torch.uint8).reshape(pages, H_kv, page, d)
    scales = byte.to(torch.uint8).expand(-1, -1, -1, BLOCK, 1).reshape(pages, H_kv, page)
    return codes.contiguous(), scales.contiguous()


def _state(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device=DEV).manual_seed(seed)
    c, s = case, {"case": case}
    n, starts = _lengths(c)
    T = int(n.sum())
    if c["op"] in ("rope", "rope_bwd"):
        s["q"] = _normal(gpu, (T, c["H"], c["d"]), _head_rms(gpu, c["H"]))
        s["k"] = _normal(gpu, (T, c["H_kv"], c["d"]), _head_rms(gpu, c["H_kv"]))
        i = torch.arange(0, c["rot"], 2, dtype=torch.float64)
        s["inv_freq"] = 10000.0 ** (-i / c["rot"]) / c["factor"]
        s["mscale"] = 1.0 + 0.1 * math.log(c["factor"])
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["inv_freq_dev"] = s["inv_freq"].to(DEV)
    elif c["op"] in ("write", "read"):
        s["table"], pages = _table(cpu, starts + n, c["page"])
        shape = (pages, c["H_kv"], c["page"])
        if c["op"] == "read" or c["ctx"]:
            s["k_codes"], s["k_scales"] = _filled(gpu, *shape, c["d"])
            s["v_codes"], s["v_scales"] = _filled(gpu, *shape, c["d"])
        else:
            s["k_codes"], s["v_codes"] = (torch.zeros(*shape, c["d"], dtype=torch.uint8, device=DEV) for _ in range(2))
            s["k_scales"], s["v_scales"] = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
        if c["op"] == "write":
            s["k"] = _normal(gpu, (T, c["H_kv"], c["d"]), _head_rms(gpu, c["H_kv"]))
            s["v"] = _normal(gpu, (T, c["H_kv"], c["d"]), _head_rms(gpu, c["H_kv"]))
        else:
            s["k_out"] = torch.empty(T, c["H_kv"], c["d"], dtype=torch.bfloat16, device=DEV)
            s["v_out"] = torch.empty_like(s["k_out"])
    else:
        lens = starts + n
        s["table"], pages = _table(cpu, lens, c["page"])
        s["k_codes"], s["k_scales"] = _filled(gpu, pages, c["H_kv"], c["page"], c["d"])
        s["v_codes"], s["v_scales"] = _filled(gpu, pages, c["H_kv"], c["page"], c["d"])
        s["q"] = _normal(gpu, (T, c["H"], c["d"]), _head_rms(gpu, c["H"]))
        s["lens"] = _int32(lens)
        s["new_max"] = int(n.max())
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(c["H"], T, dtype=torch.float32, device=DEV)
    s["T"] = T
    s["cu"], s["starts"] = _int32(_offsets(n)), _int32(starts)
    return s


def prepare(case, seed):
    s = _state(case, seed)
    if own:
        from precision_causal_attention_block_gb300 import flamia as fl
        if case["op"] in ("rope", "rope_bwd"):
            s["rotary"] = fl.Rotary(s["inv_freq"], interleaved=case["interleaved"], mscale=s["mscale"], device=DEV)
        else:
            s["cache"] = fl.KVCache.from_buffers(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                                                 token_scales=case.get("token_scales", False))
    return s


# ------------------------------------------------------------------ plain forms

def _positions(s):
    """(sequence, position) of every packed token."""
    t = torch.arange(s["T"], device=DEV)
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:], t, right=True)
    return b, s["starts"].long()[b] + t - cu[b]


def _rotated(x, cos, sin, rot, interleaved):
    x = x.float()
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y.to(torch.bfloat16)


def _rope(s):
    c = s["case"]
    _, pos = _positions(s)
    angle = pos.double()[:, None, None] * s["inv_freq_dev"]
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()
    if c["op"] == "rope_bwd":
        sin = -sin
    return tuple(_rotated(s[n], cos, sin, c["rot"], c["interleaved"]) for n in ("q", "k"))


def _slots(s):
    """(page, offset inside it) of every packed token."""
    b, pos = _positions(s)
    page = s["case"]["page"]
    return s["table"].long()[b, pos // page], pos % page


def _write_one(s, x, codes, scales):
    """Block exponents from the new tokens and what the block holds; what it
    holds is rounded again where the exponent grew."""
    c = s["case"]
    page, off = _slots(s)
    f8 = codes.view(torch.float8_e4m3fn)
    x = x.float()
    amax = x.abs().amax(2)  # [T, H_kv]
    if c["token_scales"]:
        byte = _scale_byte(amax)
        f8[page, :, off] = _codes(x, byte[:, :, None])
        scales[page, :, off] = byte.to(torch.uint8)
        return
    b, pos = _positions(s)
    starts = s["starts"].long()
    first = torch.div(s["cu"].long()[:-1], BLOCK, rounding_mode="floor") + 2 * torch.arange(c["batch"], device=DEV)
    block = first[b] + pos // BLOCK - (starts // BLOCK)[b]
    blocks = s["T"] // BLOCK + 2 * c["batch"] + 2
    most = torch.zeros(blocks, c["H_kv"], device=DEV).scatter_reduce(0, block[:, None].expand_as(amax), amax, "amax")
    byte = _scale_byte(most)  # [blocks, H_kv]
    # what the first block of each sequence holds already
    held = (starts % BLOCK > 0) & (s["cu"][1:] > s["cu"][:-1])
    lane = torch.arange(BLOCK, device=DEV)
    at = (starts // BLOCK * BLOCK)[:, None] + lane  # [B, 32]
    at_page = s["table"].long().gather(1, (at // c["page"]).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    at_off = at % c["page"]
    old_byte = scales[at_page[:, 0], :, at_off[:, 0]].to(torch.int32)  # [B, H_kv]
    byte[first] = torch.where(held[:, None], torch.maximum(byte[first], old_byte), byte[first])
    new_byte = byte[first]
    keep = held[:, None] & (at < starts[:, None])  # [B, 32]
    old = f8[at_page, :, at_off].float()  # [B, 32, H_kv, d]
    again = (old * _pow2(127 + old_byte - new_byte)[:, None, :, None]).to(torch.float8_e4m3fn)
    i, j = keep.nonzero(as_tuple=True)
    f8[at_page[i, j], :, at_off[i, j]] = again[i, j]
    scales[at_page[i, j], :, at_off[i, j]] = new_byte[i].to(torch.uint8)
    f8[page, :, off] = _codes(x, byte[block][:, :, None])
    scales[page, :, off] = byte[block].to(torch.uint8)


def _written(s):
    """The pool's codes as the values they stand for, and the scale bytes."""
    return {"k": s["k_codes"].view(torch.float8_e4m3fn), "k_scales": s["k_scales"],
            "v": s["v_codes"].view(torch.float8_e4m3fn), "v_scales": s["v_scales"]}


def _read_one(s, codes, scales):
    page, off = _slots(s)
    x = codes.view(torch.float8_e4m3fn)[page, :, off].float() * _pow2(scales[page, :, off])[:, :, None]
    return x.to(torch.bfloat16)


def _sequences(s, codes, scales):
    """The cached tokens of every sequence, float32 [B, H_kv, L, d]."""
    t = s["table"].long().clamp(min=0)
    x = codes.view(torch.float8_e4m3fn)[t].float()  # [B, pages, H_kv, page, d]
    x *= _pow2(scales[t])[..., None]
    B, n, H_kv, page, d = x.shape
    return x.transpose(1, 2).reshape(B, H_kv, n * page, d)


def _attend(s):
    c = s["case"]
    B, H, H_kv, d = c["batch"], c["H"], c["H_kv"], c["d"]
    n = s["new_max"]
    b, pos = _positions(s)
    row = torch.arange(s["T"], device=DEV) - s["cu"].long()[b]
    q = torch.zeros(B, n, H, d, device=DEV)
    q[b, row] = s["q"].float()
    q = q.view(B, n, H_kv, H // H_kv, d).permute(0, 2, 3, 1, 4).reshape(B, H_kv, -1, d)
    k = _sequences(s, s["k_codes"], s["k_scales"])
    x = (q @ k.transpose(2, 3)).view(B, H, n, -1) * d ** -0.5
    del k
    at = torch.arange(x.shape[3], device=DEV)
    here = (s["starts"].long()[:, None] + torch.arange(n, device=DEV))[:, :, None]  # [B, n, 1]
    seen = (at <= here) & (at < s["lens"].long()[:, None, None])
    if c["window"]:
        seen &= (at > here - c["window"]) | (at < c["sinks"])
    x = x.masked_fill_(~seen[:, None], -math.inf)
    m = x.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(3, keepdim=True)
    v = _sequences(s, s["v_codes"], s["v_scales"])
    o = (p.view(B, H_kv, -1, p.shape[3]) @ v).view(B, H, n, d) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log())[..., 0]
    return o[b, :, row].to(torch.bfloat16), lse[b, :, row].t().contiguous()


def _plain(s):
    op = s["case"]["op"]
    if op in ("rope", "rope_bwd"):
        return _rope(s)
    if op == "write":
        _write_one(s, s["k"], s["k_codes"], s["k_scales"])
        _write_one(s, s["v"], s["v_codes"], s["v_scales"])
        return _written(s)
    if op == "read":
        return _read_one(s, s["k_codes"], s["k_scales"]), _read_one(s, s["v_codes"], s["v_scales"])
    return _attend(s)


def run(s):
    if not own:
        return _plain(s)
    c = s["case"]
    if c["op"] in ("rope", "rope_bwd"):
        return s["rotary"](s["q"], s["k"], s["cu"], s["starts"], q_out=s["q_out"], k_out=s["k_out"],
                           inverse=c["op"] == "rope_bwd")
    if c["op"] == "write":
        s["cache"].write(s["k"], s["v"], s["cu"], s["starts"], s["table"])
        return _written(s)
    if c["op"] == "read":
        return s["cache"].read(s["cu"], s["starts"], s["table"], s["T"], k_out=s["k_out"], v_out=s["v_out"])
    return s["cache"].attend(s["q"], s["cu"], s["starts"], s["table"], c["d"] ** -0.5, window=c["window"],
                             sinks=c["sinks"], o=s["o"], lse=s["lse"])


# ------------------------------------------------------------------ work

def work(case):
    c = case
    n, starts = (x.double() for x in _lengths(c))
    T = float(n.sum())
    if c["op"] in ("rope", "rope_bwd"):
        x = T * (c["H"] + c["H_kv"])
        return {"bytes": 4 * x * c["d"], "flops": 3 * x * c["rot"]}
    if c["op"] in ("write", "read"):  # BF16 on one side, codes and a scale byte on the other
        x = 2 * T * c["H_kv"]
        return {"bytes": x * (3 * c["d"] + 1), "flops": 2 * x * c["d"]}
    lens = starts + n
    seen, cached = starts + (n + 1) / 2, lens  # keys of a mean new token; keys that any of them sees
    if c["window"]:
        most = torch.full_like(n, c["window"] + c["sinks"])
        seen, cached = torch.minimum(seen, most), torch.minimum(cached, most + n - 1)
    return {"bytes": 2 * float(cached.sum()) * c["H_kv"] * (c["d"] + 1) + T * c["H"] * (4 * c["d"] + 4),
            "flops": 4 * float((n * seen).sum()) * c["H"] * c["d"]}


# ------------------------------------------------------------------ in 64 bits

def _e4m3_values():
    """The 256 values of E4M3 codes, float64."""
    v = []
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        x = math.nan if (i & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if i & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _e8m0_values():
    return torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device=DEV)


def _two(e):
    """2^e as float64, whole e in [-300, 300]."""
    table = torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=DEV)
    return table[e.long() + 300]


def _to_e4m3(x):
    """Nearest E4M3 value, ties to even, of float64 values of at most 448."""
    _, e = torch.frexp(x)
    step = _two((e - 1).clamp(-6, 8) - 3)
    return (x / step).round() * step


def _exact_rope(s):
    c, out = s["case"], []
    w = s["inv_freq_dev"]
    cu, starts = s["cu"].tolist(), s["starts"].tolist()
    pos = torch.cat([torch.arange(a, a + e - b, device=DEV) for a, b, e in zip(starts, cu, cu[1:])])
    turn = torch.polar(torch.full((s["T"], 1, w.numel()), s["mscale"], dtype=torch.float64, device=DEV),
                       pos.double()[:, None, None] * w)
    if c["op"] == "rope_bwd":
        turn = turn.conj()
    for n in ("q", "k"):
        x = s[n].double()
        r = x[..., :c["rot"]]
        pair = r.unflatten(2, (-1, 2)) if c["interleaved"] else r.unflatten(2, (2, -1)).transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z.flatten(2) if c["interleaved"] else z.transpose(2, 3).flatten(2)
        out.append(torch.cat([z, x[..., c["rot"]:]], 2))
    return tuple(out)


def _exact_write(s, x, codes, scales, value, power):
    """The pool's code values after the write, sequence by sequence."""
    c = s["case"]
    page = c["page"]
    pool = value[codes.long()]
    cu, starts = s["cu"].tolist(), s["starts"].tolist()
    table = s["table"].long()
    for b in range(c["batch"]):
        n, a = cu[b + 1] - cu[b], starts[b]
        if n == 0:
            continue
        new = x[cu[b]:cu[b + 1]].double()
        lead = 0 if c["token_scales"] else a % BLOCK
        at = torch.arange(a - lead, a + n, device=DEV)
        pg, off = table[b, at // page], at % page
        held = pool[pg[:lead], :, off[:lead]]
        size = 1 if c["token_scales"] else BLOCK
        tail = -(lead + n) % size
        top = torch.cat([new.new_zeros(lead, c["H_kv"]), new.abs().amax(2), new.new_zeros(tail, c["H_kv"])])
        top = top.view(-1, size, c["H_kv"]).amax(1)
        e = torch.full(top.shape, -127.0, dtype=torch.float64, device=DEV)
        e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448)), e)
        e = torch.where(448 * _two(e - 1) >= top, e - 1, e)  # log2 next to a border
        e = torch.where(448 * _two(e) < top, e + 1, e).clamp(-127, 127)
        if lead:
            was = scales[pg[0], :, off[0]].double() - 127
            e[0] = torch.maximum(e[0], was)
            pool[pg[:lead], :, off[:lead]] = _to_e4m3(held * _two(was - e[0])[:, None])
        e = e.repeat_interleave(size, 0)[lead:lead + n]
        pool[pg[lead:], :, off[lead:]] = _to_e4m3(new * _two(-e)[:, :, None])
    return pool


def _exact_tokens(s, b, n, codes, scales, value, power):
    """The first n cached tokens of sequence b, float64 [n, H_kv, d]."""
    at = torch.arange(n, device=DEV)
    pg, off = s["table"].long()[b, at // s["case"]["page"]], at % s["case"]["page"]
    return value[codes[pg, :, off].long()] * power[scales[pg, :, off].long()][:, :, None]


def exact(case, seed):
    s = _state(case, seed)
    value, power = _e4m3_values(), _e8m0_values()
    c = case
    if c["op"] in ("rope", "rope_bwd"):
        return _exact_rope(s)
    if c["op"] == "write":
        return {"k": _exact_write(s, s["k"], s["k_codes"], s["k_scales"], value, power), "k_scales": None,
                "v": _exact_write(s, s["v"], s["v_codes"], s["v_scales"], value, power), "v_scales": None}
    cu, starts = s["cu"].tolist(), s["starts"].tolist()
    if c["op"] == "read":
        both = []
        for n in ("k", "v"):
            both.append(torch.cat([_exact_tokens(s, b, starts[b] + cu[b + 1] - cu[b], s[n + "_codes"], s[n + "_scales"],
                                                 value, power)[starts[b]:] for b in range(c["batch"])]))
        return tuple(both)
    o = torch.zeros(s["T"], c["H"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["H"], s["T"], dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        n = cu[b + 1] - cu[b]
        L = starts[b] + n
        k = _exact_tokens(s, b, L, s["k_codes"], s["k_scales"], value, power)
        v = _exact_tokens(s, b, L, s["v_codes"], s["v_scales"], value, power)
        i = torch.arange(starts[b], L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)
        seen = j <= i
        if c["window"]:
            seen &= (j > i - c["window"]) | (j < c["sinks"])
        for h in range(c["H"]):
            g = h // (c["H"] // c["H_kv"])
            x = s["q"][cu[b]:cu[b + 1], h].double() @ k[:, g].t() / math.sqrt(c["d"])
            x = torch.where(seen, x, x.new_full((), -math.inf))
            lse[h, cu[b]:cu[b + 1]] = torch.logsumexp(x, 1)
            o[cu[b]:cu[b + 1], h] = torch.softmax(x, 1) @ v[:, g]
    return o, lse
