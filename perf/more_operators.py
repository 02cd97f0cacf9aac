"""Workloads of many continuations of one prompt: what is timed, and what each
result is compared with.

Five operators around the paged MXFP8 cache:

* ``rope`` / ``rope_bwd``: rotary positions with several axes (time, height,
  width) of Q and K, and of dQ and dK;
* ``copy``: pages of the cache copied to other pages;
* ``fork``: sequences that continue others share their pages, and those that
  are about to be written get pages of their own;
* ``compact``: pages that are in use moved to the front of the pool;
* ``attend``: attention of new tokens over the cache where the sequences of a
  batch share a long prefix, which is read once for all of them.

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
        # one decode step of 16 sequences that look at images: latency
        {"name": "rope_decode", "op": "rope", "batch": 16, "lo": 1, "hi": 1, "H": 32, "H_kv": 8, "d": 128,
         "rot": 128, "sections": "16,24,24", "cyclic": False, "interleaved": False, "factor": 1.0, "ctx": 131072},
        # dQ and dK of a long video's training call
        {"name": "rope_bwd_video", "op": "rope_bwd", "batch": 1, "lo": 131072, "hi": 131072, "H": 32, "H_kv": 32, "d": 64,
         "rot": 64, "sections": "8,12,12", "cyclic": True, "interleaved": True, "factor": 4.0, "ctx": 0},
        # a handful of pages to the pages of another sequence: latency
        {"name": "copy_few", "op": "copy", "pages": 7, "H_kv": 4, "d": 64, "page": 32},
        # the contexts of a serving batch taken to another part of the pool
        {"name": "copy_many", "op": "copy", "pages": 4099, "H_kv": 8, "d": 128, "page": 64},
        # eight answers to one question, about to write their first token: latency
        {"name": "fork_one", "op": "fork", "prompts": 1, "branches": 8, "ctx_lo": 517, "ctx_hi": 517, "H_kv": 4, "d": 64,
         "page": 64, "new": 1},
        # four beams of each of 48 long prompts, large pages
        {"name": "fork_beams", "op": "fork", "prompts": 48, "branches": 4, "ctx_lo": 1000, "ctx_hi": 16384, "H_kv": 16,
         "d": 128, "page": 128, "new": 1},
        # a small pool after most of its sequences ended
        {"name": "compact_small", "op": "compact", "batch": 6, "lo": 33, "hi": 700, "H_kv": 4, "d": 64, "page": 32,
         "spare": 1.5},
        # a serving pool, half of it in use
        {"name": "compact_pool", "op": "compact", "batch": 96, "lo": 16, "hi": 16384, "H_kv": 8, "d": 128, "page": 64,
         "spare": 1.0},
        # eight answers over a system prompt: latency
        {"name": "attend_few", "op": "attend", "batch": 8, "idle": 0, "new": 1, "prefix": 2048, "own_lo": 1, "own_hi": 130,
         "H": 16, "H_kv": 16, "d": 128, "page": 64},
        # a serving batch over one long document, grouped heads, ragged answers
        {"name": "attend_batch", "op": "attend", "batch": 96, "idle": 7, "new": 1, "prefix": 16421, "own_lo": 1,
         "own_hi": 2048, "H": 32, "H_kv": 8, "d": 128, "page": 64},
        # questions about the longest training context
        {"name": "attend_long", "op": "attend", "batch": 24, "idle": 0, "new": 1, "prefix": 131072, "own_lo": 16,
         "own_hi": 512, "H": 32, "H_kv": 32, "d": 64, "page": 256},
        # drafted tokens of many answers
        {"name": "attend_drafts", "op": "attend", "batch": 128, "idle": 0, "new": 4, "prefix": 8191, "own_lo": 4,
         "own_hi": 1024, "H": 16, "H_kv": 4, "d": 128, "page": 32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "copy", "fork", "compact", "attend", "attend", "attend"])
    d = rng.choice([64, 128])
    H_kv = rng.choice([1, 2, 4, 5, 8, 16])
    H = H_kv * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * H_kv <= 32])
    page = rng.choice([32, 64, 128, 256])
    if op in ("rope", "rope_bwd"):
        batch = _log(rng, 1, 96)
        n = max(1, _log(rng, 1, 65536) // batch)
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
        axes = rng.choice([1, 2, 3, 3, 4])
        cuts = sorted(rng.randint(0, rot // 2) for _ in range(axes - 1))
        parts = [b - a for a, b in zip([0] + cuts, cuts + [rot // 2])]
        return {"op": op, "batch": batch, "lo": max(1, n // 2), "hi": n, "H": H, "H_kv": H_kv, "d": d, "rot": rot,
                "sections": ",".join(str(p) for p in parts), "cyclic": rng.random() < 0.5,
                "interleaved": rng.random() < 0.5, "factor": rng.choice([1.0, 4.0, 8.0]),
                "ctx": rng.choice([0, _log(rng, 1, 131072)])}
    most = int(2.5e8 / (H_kv * d))  # cached tokens of a drawn pool
    if op == "copy":
        return {"op": op, "pages": _log(rng, 1, max(1, most // page)), "H_kv": H_kv, "d": d, "page": page}
    if op == "fork":
        m, k = _log(rng, 1, 64), _log(rng, 1, 32)
        hi = max(1, min(_log(rng, 1, 16384), most // m, 60000 * page // (m * k + 1)))
        return {"op": op, "prompts": m, "branches": k, "ctx_lo": max(1, hi // 3), "ctx_hi": hi, "H_kv": H_kv, "d": d,
                "page": page, "new": rng.choice([1, 1, 5, 40])}
    if op == "compact":
        batch = _log(rng, 1, 96)
        hi = max(1, min(_log(rng, 1, 16384), most // batch))
        return {"op": op, "batch": batch, "lo": max(1, hi // 8), "hi": hi, "H_kv": H_kv, "d": d, "page": page,
                "spare": rng.choice([0.1, 0.5, 1.0, 3.0])}
    batch, new = _log(rng, 2, 128), rng.choice([1, 1, 1, 2, 4])
    prefix = min(_log(rng, 256, 131072), most)
    tail = max(new, min(_log(rng, 1, 2048), most // batch))
    prefix = max(256, min(prefix, int(1.2e8 / (batch * new * H))))
    return {"op": op, "batch": batch, "idle": rng.choice([0, 0, 3, 11]), "new": new, "prefix": prefix,
            "own_lo": max(new, tail // 8), "own_hi": tail, "H": H, "H_kv": H_kv, "d": d, "page": page}


# ------------------------------------------------------------------ inputs

def _case_generator(case):
    """Whole numbers that belong to a case, whatever the seed."""
    return torch.Generator().manual_seed(zlib.crc32(json.dumps(
        {k: v for k, v in case.items() if k != "name"}, sort_keys=True).encode()))


def _between(gen, n, lo, hi):
    """n whole numbers in [lo, hi], spread over their logarithm where that is wide."""
    u = torch.rand(n, generator=gen, dtype=torch.float64)
    if hi > 10 * lo:
        x = torch.exp(math.log(max(lo, 1)) + u * (math.log(hi) - math.log(max(lo, 1)))).round()
    else:
        x = lo + (u * (hi - lo + 1)).floor()
    return x.clamp(lo, hi).to(torch.int64)


def _offsets(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])


def _int32(x):
    return x.to(torch.int32).to(DEV)


def _normal(gen, shape, rms):
    return (torch.randn(shape, generator=gen, device=DEV) * rms).to(torch.bfloat16)


def _head_rms(gen, H):
    """Per-head RMS in [0.5, 2], as in the training workloads."""
    return 0.5 + 1.5 * torch.rand(H, generator=gen, device=DEV)[:, None]


def _pow2(byte):
    """2^(byte - 127) as float32, from E8M0 bytes."""
    b = byte.to(torch.int32)
    return torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)


def _pool(gen, pages, H_kv, page, d):
    """Pages as a block-scaled write leaves them: (codes, scale bytes)."""
    x = _normal(gen, (pages, H_kv, page, d), _head_rms(gen, H_kv)[None, :, :, None]).float()
    x = x.view(pages, H_kv, page // BLOCK, BLOCK, d)
    m, e = torch.frexp(x.abs().amax((3, 4), keepdim=True))
    byte = torch.where(m <= 0.875, e - 9, e - 8) + 127  # the largest element below 448 2^(byte - 127)
    codes = (x * _pow2(254 - byte)).to(torch.float8_e4m3fn).view(torch.uint8).reshape(pages, H_kv, page, d)
    scales = byte.to(torch.uint8).expand(-1, -1, -1, BLOCK, 1).reshape(pages, H_kv, page)
    return codes.contiguous(), scales.contiguous()


def _pools(s, gen, pages, c):
    for n in ("k", "v"):
        s[n + "_codes"], s[n + "_scales"] = _pool(gen, pages, c["H_kv"], c["page"], c["d"])


def _table(order, lens, page, width):
    """Page table of sequences of these lengths over pages taken from `order` in turn;
    -1 where a sequence has none."""
    need = (lens + page - 1) // page
    first = _offsets(need)
    slot = torch.arange(width)
    at = first[:-1, None] + slot
    return torch.where(slot < need[:, None], order[at.clamp(max=order.numel() - 1)], torch.full_like(at, -1))


def _positions(lens, starts, axes, gen):
    """[axes, T] positions of packed sequences: text, where all axes go on together,
    and pictures of 24 x 36 patches a time step."""
    out = []
    for n, a in zip(lens.tolist(), starts.tolist()):
        u = torch.arange(n)
        text = min(n, int(torch.randint(0, 64, (1,), generator=gen)))
        v = (u - text).clamp(min=0)
        coords = [v // 864, v // 36 % 24, v % 36, v // 12 % 3][:axes]
        out.append(torch.stack([torch.where(u < text, u, text + x) + a for x in coords]))
    return torch.cat(out, 1)


def _sections(c):
    return [int(x) for x in c["sections"].split(",")]


def _pair_axes(c):
    """The axis of every pair: sections one behind the other, or by turns."""
    left = _sections(c)
    if not c["cyclic"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _shared_lengths(c):
    """(new tokens, tokens cached in all) of an attend case's sequences."""
    tail = _between(_case_generator(c), c["batch"], c["own_lo"], c["own_hi"])
    n = torch.full_like(tail, c["new"])
    if c["idle"]:
        n[::c["idle"]] = 0
    return n, torch.where(n > 0, c["prefix"] + tail, torch.zeros_like(tail))


def _compact_layout(c):
    """(page table, uses of each page) of a pool whose pages are handed out in random
    order; every third sequence shares the first half of the pages of the one before."""
    gen = _case_generator(c)
    lens = _between(gen, c["batch"], c["lo"], c["hi"])
    need = (lens + c["page"] - 1) // c["page"]
    pages = int(int(need.sum()) * (1 + c["spare"])) + 1
    table = _table(torch.randperm(pages, generator=gen), lens, c["page"], int(need.max()))
    for b in range(2, c["batch"], 3):
        half = int(min(need[b], need[b - 1])) // 2
        table[b, :half] = table[b - 1, :half]
    refs = torch.bincount(table[table >= 0], minlength=pages)
    return table, refs


def _state(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device=DEV).manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] in ("rope", "rope_bwd"):
        gen = _case_generator(c)
        n = _between(gen, c["batch"], c["lo"], c["hi"])
        starts = torch.randint(0, c["ctx"] + 1, (c["batch"],), generator=cpu)
        T = int(n.sum())
        s["cu"], s["pos"] = _int32(_offsets(n)), _int32(_positions(n, starts, len(_sections(c)), cpu))
        s["q"] = _normal(gpu, (T, c["H"], c["d"]), _head_rms(gpu, c["H"]))
        s["k"] = _normal(gpu, (T, c["H_kv"], c["d"]), _head_rms(gpu, c["H_kv"]))
        i = torch.arange(0, c["rot"], 2, dtype=torch.float64)
        s["inv_freq"] = 10000.0 ** (-i / c["rot"]) / c["factor"]
        s["inv_freq_dev"] = s["inv_freq"].to(DEV)
        s["axis_dev"] = torch.tensor(_pair_axes(c), device=DEV)
        s["mscale"] = 1.0 + 0.1 * math.log(c["factor"])
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    elif c["op"] == "copy":
        n = c["pages"]
        _pools(s, gpu, 2 * n + 3, c)
        order = torch.randperm(2 * n + 3, generator=cpu)
        s["src"], s["dst"] = _int32(order[:n]), _int32(order[n:2 * n])
    elif c["op"] == "fork":
        m, k, page = c["prompts"], c["branches"], c["page"]
        lens = torch.cat([_between(_case_generator(c), m, c["ctx_lo"], c["ctx_hi"]),
                          torch.zeros(m * k, dtype=torch.int64)])
        width = (int(lens.max()) + c["new"]) // page + 1
        used = int(((lens + page - 1) // page).sum())
        pages = used + m * k * (c["new"] // page + 2)
        order = torch.randperm(pages, generator=cpu)
        table = _table(order, lens, page, width)
        refs = torch.zeros(pages, dtype=torch.int64)
        refs[order[:used]] = 1
        _pools(s, gpu, pages, c)
        s["table"], s["refs"], s["lens"] = _int32(table), _int32(refs), _int32(lens)
        s["parents"] = _int32(torch.arange(m).repeat_interleave(k))
        s["children"] = _int32(m + torch.arange(m * k))
        s["cu"] = _int32(_offsets((torch.arange(m + m * k) >= m) * c["new"]))
    elif c["op"] == "compact":
        table, refs = _compact_layout(c)
        _pools(s, gpu, refs.numel(), c)
        s["table0"], s["refs0"] = _int32(table), _int32(refs)
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
    else:
        n, lens = _shared_lengths(c)
        page, P = c["page"], c["prefix"]
        whole = P // page  # pages that all sequences share
        mine = torch.where(n > 0, lens - whole * page, torch.zeros_like(lens))
        pages = whole + int(((mine + page - 1) // page).sum()) + 1
        order = torch.randperm(pages, generator=cpu)
        tail = _table(order[whole:], mine, page, max(1, int((mine + page - 1).max()) // page))
        head = order[:whole].expand(c["batch"], whole)
        table = torch.cat([torch.where((n > 0)[:, None], head, torch.full_like(head, -1)), tail], 1)
        _pools(s, gpu, pages, c)
        s["table"] = _int32(table)
        busy = (n > 0).nonzero()[:, 0]
        if P % page:  # the page in which the prefix ends is copied by each of them
            at = s["table"][busy.to(DEV), whole].long()
            for x in ("k_codes", "k_scales", "v_codes", "v_scales"):
                s[x][at[1:], :, :P % page] = s[x][at[0], :, :P % page].clone()
        T = int(n.sum())
        s["q"] = _normal(gpu, (T, c["H"], c["d"]), _head_rms(gpu, c["H"]))
        s["cu"], s["starts"], s["lens"] = _int32(_offsets(n)), _int32(lens - n), _int32(lens)
        s["busy"], s["tail"] = busy.to(DEV), int((lens - n).max()) + c["new"] - P
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(c["H"], T, dtype=torch.float32, device=DEV)
    return s


def prepare(case, seed):
    s = _state(case, seed)
    if own:
        from precision_causal_attention_block_gb300 import flamia as fl
        if case["op"] in ("rope", "rope_bwd"):
            s["rotary"] = fl.Rotary(s["inv_freq"], interleaved=case["interleaved"], mscale=s["mscale"], device=DEV,
                                    axes=fl.rope_axes(_sections(case), cyclic=case["cyclic"]))
        else:
            s["cache"] = fl.KVCache.from_buffers(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        if case["op"] in ("fork", "compact"):
            s["pool"] = fl.PagePool.from_buffers(s["cache"], s["table"], s["refs"])
    return s


# ------------------------------------------------------------------ plain forms

def _rope(s):
    c = s["case"]
    angle = s["pos"].double()[s["axis_dev"]].t()[:, None] * s["inv_freq_dev"]  # [T, 1, pairs]
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()
    if c["op"] == "rope_bwd":
        sin = -sin
    out, r = [], c["rot"]
    for n in ("q", "k"):
        x = s[n].float()
        y = x.clone()
        first = slice(0, r, 2) if c["interleaved"] else slice(0, r // 2)
        second = slice(1, r, 2) if c["interleaved"] else slice(r // 2, r)
        a, b = x[..., first], x[..., second]
        y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
        out.append(y.to(torch.bfloat16))
    return tuple(out)


def _contents(s):
    """The pool's codes as the values they stand for, and the scale bytes."""
    return {"k": s["k_codes"].view(torch.float8_e4m3fn), "k_scales": s["k_scales"],
            "v": s["v_codes"].view(torch.float8_e4m3fn), "v_scales": s["v_scales"]}


POOL = ("k_codes", "k_scales", "v_codes", "v_scales")


def _copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for n in POOL:
        s[n][dst] = s[n][src]
    return _contents(s)


def _counted(refs, pages, by):
    """refs + by at every page of `pages` (negative ones: none)."""
    p = pages.reshape(-1).long()
    more = torch.where(p >= 0, torch.full_like(p, by), torch.zeros_like(p)).to(refs.dtype)
    refs.index_add_(0, p.clamp(min=0), more)


def _fork(s):
    """Children give their pages back and take their parents' (fork); then every
    sequence gets pages for its new tokens, the free ones in order, and a copy of a
    page that others use as well (reserve)."""
    c, table, refs, lens = s["case"], s["table"], s["refs"], s["lens"]
    page = c["page"]
    par, chi = s["parents"].long(), s["children"].long()
    slot = torch.arange(table.shape[1], device=DEV)
    held = (lens[par] + page - 1) // page
    rows = torch.where(slot < held[:, None], table[par], torch.full_like(table[par], -1))
    _counted(refs, table[chi], -1)
    _counted(refs, rows, 1)
    table[chi], lens[chi] = rows, lens[par]
    # pages of the new tokens
    n = s["cu"][1:] - s["cu"][:-1]
    j0, j1 = lens // page, (lens + n - 1) // page
    wanted = (slot >= j0[:, None]) & (slot <= j1[:, None]) & (n > 0)[:, None]
    have = wanted & (table >= 0)
    at = table.long().clamp(min=0)
    many = have & (refs[at] > 1)
    here = torch.zeros_like(refs).index_add_(0, at.reshape(-1), many.reshape(-1).to(refs.dtype))
    order = torch.arange(table.numel(), device=DEV).view_as(table)
    last = torch.full(refs.shape, -1, device=DEV).scatter_reduce(
        0, at.reshape(-1), torch.where(many, order, torch.full_like(order, -1)).reshape(-1), "amax")
    keeps = many & (here[at] == refs[at]) & (last[at] == order)  # the last of a page's users keeps it
    moves = many & ~keeps
    need = (wanted & (table < 0)) | moves
    free = torch.sort((refs != 0).to(torch.int8), stable=True)[1]
    new = free[(need.reshape(-1).cumsum(0) - 1).clamp(min=0, max=refs.numel() - 1)].view_as(table)
    b, j = (moves & (slot == j0[:, None])).nonzero(as_tuple=True)
    src, dst = at[b, j], new[b, j]
    keep = torch.arange(page, device=DEV) < (lens[b] % page)[:, None]
    for x in POOL:
        m = keep[:, None, :, None] if s[x].dim() == 4 else keep[:, None, :]
        s[x][dst] = torch.where(m, s[x][src], s[x][dst])
    _counted(refs, torch.where(moves, table, torch.full_like(table, -1)), -1)
    table.copy_(torch.where(need, new.to(table.dtype), table))
    _counted(refs, torch.where(need, table, torch.full_like(table, -1)), 1)
    return {**_contents(s), "table": table, "refs": refs, "lens": lens}


def _compact(s):
    """The k-th used page behind the first `live` ones goes to the k-th free page
    among them."""
    table, refs = s["table"], s["refs"]
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    used = refs > 0
    live = used.sum()
    i = torch.arange(refs.numel(), device=DEV)
    src, dst = (used & (i >= live)).nonzero()[:, 0], (~used & (i < live)).nonzero()[:, 0]
    for n in POOL:
        s[n][dst] = s[n][src]
    to = i.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].to(table.dtype), table))
    return {**_contents(s), "table": table, "refs": refs, "live": live.to(torch.int32).view(1)}


def _rows(s, n, pages, first, count):
    """Tokens first .. first + count - 1 of sequences with these page-table rows,
    float32 [B, H_kv, count, d]."""
    page = s["case"]["page"]
    at = first + torch.arange(count, device=DEV)
    pg = pages[:, (at // page).clamp(max=pages.shape[1] - 1)].clamp(min=0)  # [B, count]
    x = s[n + "_codes"].view(torch.float8_e4m3fn)[pg, :, at % page].float()
    x *= _pow2(s[n + "_scales"][pg, :, at % page])[..., None]
    return x.transpose(1, 2)


def _attend(s):
    c = s["case"]
    B, n, H, H_kv, d, P = s["busy"].numel(), c["new"], c["H"], c["H_kv"], c["d"], c["prefix"]
    G = H // H_kv
    pages = s["table"].long()[s["busy"]]
    q = s["q"].float().view(B, n, H_kv, G, d).permute(2, 0, 3, 1, 4)  # [H_kv, B, G, n, d]
    head = _rows(s, "k", pages[:1], 0, P)[0]
    x0 = q.reshape(H_kv, -1, d) @ head.transpose(1, 2)  # [H_kv, B G n, P]
    x0 = x0.view(H_kv, B, G * n, P) * d ** -0.5
    tail = _rows(s, "k", pages, P, s["tail"]).transpose(0, 1)  # [H_kv, B, tail, d]
    x1 = (q.reshape(H_kv, B, G * n, d) @ tail.transpose(2, 3)).view(H_kv, B, G, n, -1) * d ** -0.5
    at = P + torch.arange(s["tail"], device=DEV)
    here = s["starts"].long()[s["busy"], None] + torch.arange(n, device=DEV)
    x1 = x1.masked_fill(at > here[None, :, None, :, None], -math.inf).view(H_kv, B, G * n, -1)
    m = torch.maximum(x0.amax(3, keepdim=True), x1.amax(3, keepdim=True))
    x0, x1 = x0.sub_(m).exp_(), x1.sub_(m).exp_()
    l = x0.sum(3, keepdim=True) + x1.sum(3, keepdim=True)
    o = (x0.view(H_kv, -1, P) @ _rows(s, "v", pages[:1], 0, P)[0]).view(H_kv, B, G * n, d)
    o = (o + x1 @ _rows(s, "v", pages, P, s["tail"]).transpose(0, 1)) / l
    o = o.view(H_kv, B, G, n, d).permute(1, 3, 0, 2, 4).reshape(-1, H, d)
    lse = (m + l.log()).view(H_kv, B, G, n).permute(0, 2, 1, 3).reshape(H, -1)
    return o.to(torch.bfloat16), lse


def run(s):
    c = s["case"]
    if not own:
        return {"rope": _rope, "rope_bwd": _rope, "copy": _copy, "fork": _fork, "compact": _compact,
                "attend": _attend}[c["op"]](s)
    if c["op"] in ("rope", "rope_bwd"):
        return s["rotary"](s["q"], s["k"], s["cu"], positions=s["pos"], q_out=s["q_out"], k_out=s["k_out"],
                           inverse=c["op"] == "rope_bwd")
    if c["op"] == "copy":
        s["cache"].copy_pages(s["src"], s["dst"])
        return _contents(s)
    if c["op"] == "fork":
        s["pool"].fork(s["parents"], s["children"], s["lens"])
        s["pool"].reserve(s["cu"], s["lens"])
        return {**_contents(s), "table": s["table"], "refs": s["refs"], "lens": s["lens"]}
    if c["op"] == "compact":
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        live = s["pool"].compact()
        return {**_contents(s), "table": s["table"], "refs": s["refs"], "live": live}
    return s["cache"].attend(s["q"], s["cu"], s["starts"], s["table"], c["d"] ** -0.5, prefix=c["prefix"], o=s["o"],
                             lse=s["lse"])


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] in ("rope", "rope_bwd"):
        T = float(_between(_case_generator(c), c["batch"], c["lo"], c["hi"]).sum())
        x = T * (c["H"] + c["H_kv"])
        return {"bytes": 4 * x * c["d"] + 4 * T * len(_sections(c)), "flops": 3 * x * c["rot"]}
    row = 2 * c["H_kv"] * (c["d"] + 1)  # bytes of a cached token
    if c["op"] == "copy":
        return {"bytes": 2 * c["pages"] * (c["page"] * row + 4), "flops": 0}
    if c["op"] == "fork":
        lens = _between(_case_generator(c), c["prompts"], c["ctx_lo"], c["ctx_hi"])
        held = (lens + c["page"] - 1) // c["page"]
        copied = c["branches"] * float((lens % c["page"]).sum())
        new = c["branches"] * float((lens + c["new"]).sum()) / c["page"]
        return {"bytes": 2 * copied * row + 4 * (1 + 4 * c["branches"]) * float(held.sum()) + 8 * new, "flops": 0}
    if c["op"] == "compact":
        table, refs = _compact_layout(c)
        live = int((refs > 0).sum())
        moved = float((refs[live:] > 0).sum())
        return {"bytes": 2 * moved * c["page"] * row + 8 * table.numel() + 8 * refs.numel(), "flops": 0}
    n, lens = (x.double() for x in _shared_lengths(c))
    rows = float(n.sum()) * c["H"]
    cached = c["prefix"] + float((lens - c["prefix"]).clamp(min=0).sum())
    return {"bytes": cached * row + rows * (4 * c["d"] + 4),
            "flops": 4 * float((n * (lens - (n - 1) / 2)).sum()) * c["H"] * c["d"]}


# ------------------------------------------------------------------ in 64 bits

def _e4m3_values():
    """The 256 values of E4M3 codes, float64."""
    v = []
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        x = math.nan if (i & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if i & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _exact_rope(s):
    c, out = s["case"], []
    turn = torch.empty(s["q"].shape[0], c["rot"] // 2, dtype=torch.complex128, device=DEV)
    sign = -1.0 if c["op"] == "rope_bwd" else 1.0
    for pair, (axis, w) in enumerate(zip(_pair_axes(c), s["inv_freq"].tolist())):
        turn[:, pair] = torch.exp(1j * sign * w * s["pos"][axis].double()) * s["mscale"]
    for n in ("q", "k"):
        x = s[n].double()
        r = x[..., :c["rot"]]
        pair = r.unflatten(2, (-1, 2)) if c["interleaved"] else r.unflatten(2, (2, -1)).transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
        z = z.flatten(2) if c["interleaved"] else z.transpose(2, 3).flatten(2)
        out.append(torch.cat([z, x[..., c["rot"]:]], 2))
    return tuple(out)


def _exact_moves(c, s):
    """(source page, target page, rows) of what an operator copies, page by page."""
    page = c.get("page")
    if c["op"] == "copy":
        return [(a, b, page) for a, b in zip(s["src"].tolist(), s["dst"].tolist())]
    if c["op"] == "compact":
        refs = s["refs0"].tolist()
        live = sum(r > 0 for r in refs)
        holes = (p for p in range(live) if refs[p] == 0)
        return [(p, next(holes), page) for p in range(live, len(refs)) if refs[p] > 0]
    # fork: the children one after another take the lowest free pages
    table, refs, lens = s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    free = (p for p in range(len(refs)) if refs[p] == 0)
    moves = []
    for a in s["parents"].tolist():
        part = lens[a] % page
        new = (lens[a] + c["new"] - 1) // page - lens[a] // page + 1
        got = [next(free) for _ in range(new)]
        if part:
            moves.append((table[a][lens[a] // page], got[0], part))
    return moves


def _exact_pool(c, s):
    value = _e4m3_values()
    out = {}
    moves = _exact_moves(c, s)
    for n in ("k", "v"):
        x = value[s[n + "_codes"].long()]
        first = x.clone() if c["op"] == "fork" else x
        for a, b, rows in moves:  # (a source is never a target)
            x[b, :, :rows] = first[a, :, :rows]
        out[n], out[n + "_scales"] = x, None
    if c["op"] == "fork":
        out.update(table=None, refs=None, lens=None)
    if c["op"] == "compact":
        out.update(table=None, refs=None, live=None)
    return out


def exact(case, seed):
    s = _state(case, seed)
    c = case
    if c["op"] in ("rope", "rope_bwd"):
        return _exact_rope(s)
    if c["op"] in ("copy", "fork", "compact"):
        return _exact_pool(c, s)
    value = _e4m3_values()
    power = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device=DEV)
    table, cu, starts = s["table"].long(), s["cu"].tolist(), s["starts"].tolist()

    def tokens(n, b, first, end):
        at = torch.arange(first, end, device=DEV)
        pg, off = table[b, at // c["page"]], at % c["page"]
        x = value[s[n + "_codes"][pg, :, off].long()] * power[s[n + "_scales"][pg, :, off].long()][:, :, None]
        return x.transpose(0, 1)  # [H_kv, tokens, d]

    G, P = c["H"] // c["H_kv"], c["prefix"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    head = None
    for b in range(c["batch"]):
        if cu[b + 1] == cu[b]:
            continue
        end = starts[b] + cu[b + 1] - cu[b]
        if head is None:
            head = {n: tokens(n, b, 0, P) for n in ("k", "v")}
        k, v = ({n: torch.cat([head[n], tokens(n, b, P, end)], 1) for n in ("k", "v")}[x] for x in ("k", "v"))
        seen = torch.arange(end, device=DEV) <= torch.arange(starts[b], end, device=DEV)[:, None]
        for h in range(c["H"]):
            x = s["q"][cu[b]:cu[b + 1], h].double() @ k[h // G].t() / math.sqrt(c["d"])
            x = torch.where(seen, x, x.new_full((), -math.inf))
            lse[h, cu[b]:cu[b + 1]] = torch.logsumexp(x, 1)
            o[cu[b]:cu[b + 1], h] = torch.softmax(x, 1) @ v[h // G]
    return o, lse
