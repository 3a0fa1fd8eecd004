"""More operators measured on one GPU: attention of many new tokens per request over the
paged cache, scores with a tanh cap and a distance bias, and pages of 4 bits (append,
attention of one token, rows read back).

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or,
with ``own`` set, by the calls a user makes of this package.  ``exact`` gives the same
outputs from the definitions in 64 bits.

The paged cache holds, per layer, pages [n_pages, 2, h_kv, page, d]: page p's keys (index
0) and values (index 1) of ``page`` consecutive positions of one request.  Position n of
request r sits in page table[r, n // page], row n % page.  Eight-bit pages hold value /
scale with one scale per kv head for keys and one for values.

Four-bit pages are bytes [n_pages, 2, h_kv, page / 16, 9 d]: 16 positions of a head together.
Each 16 elements b of a row have one e4m3 scale s = max|x| / 7, and 4-bit codes
c = round(x / s) + 8 of x = value / scale; element e of a row is the low half of a byte where e
is even, the high half where it is odd.
  keys:   codes [position][d / 2 bytes], then scales [position][d / 16]
  values: codes [d / 32][position][16 bytes], then scales [d / 16][position]
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "int4": torch.uint8}
E4M3_MAX = 448.0
UNIT = 16          # positions, and elements of a scale


def listed():
    gqa = dict(heads=32, kv_heads=8, dim=128)
    none = dict(window=0, cap=0.0, bias=False, prefix=False)
    return [
        # a few drafted tokens checked at once behind the one-request 4K workload: latency
        dict(name="attend_draft_4k", kind="attend", req=1, lo=4091, hi=4091, new_lo=5, new_hi=5, heads=8, kv_heads=1, dim=128,
             page=64, type="bf16", kv="bf16", spread=1, **{**none, "cap": 30.0}),
        # a long prompt of a model that caps its scores
        dict(name="attend_prompt_8k", kind="attend", req=1, lo=0, hi=0, new_lo=8192, new_hi=8192, **gqa, page=64, type="bf16",
             kv="bf16", spread=2, **{**none, "cap": 50.0}),
        # ragged prompts packed into one call, some requests without a token: distance bias, prefixes seen from both sides
        dict(name="attend_prefix_ragged", kind="attend", req=24, lo=0, hi=500, new_lo=0, new_hi=900, heads=24, kv_heads=8, dim=64,
             page=16, type="fp16", kv="fp16", spread=3, **{**none, "bias": True, "prefix": True}),
        # chunks of prompts on wide heads within a sliding window
        dict(name="attend_window_wide", kind="attend", req=5, lo=0, hi=2000, new_lo=501, new_hi=1777, heads=16, kv_heads=2, dim=256,
             page=64, type="bf16", kv="bf16", spread=4, **{**none, "window": 1000}),
        # chunks of two long prompts over a cache in 4 bits
        dict(name="attend_chunk_4bit", kind="attend", req=2, lo=30000, hi=30000, new_lo=512, new_hi=512, **gqa, page=64, type="bf16",
             kv="int4", spread=5, **none),
        # one decode step of the batch-16 workload with capped scores
        dict(name="decode_cap_batch16", kind="decode", req=16, lo=32768, hi=32768, **gqa, page=64, type="bf16", kv="bf16",
             spread=6, **{**none, "cap": 50.0}),
        # requests of mixed lengths, empty ones among them, half-width heads in groups of three, distance bias
        dict(name="decode_bias_ragged", kind="decode", req=33, lo=0, hi=9001, heads=12, kv_heads=4, dim=64, page=16, type="fp16",
             kv="fp16", spread=7, **{**none, "bias": True}),
        # the batch-16 workload over 4-bit pages
        dict(name="decode_batch16_4bit", kind="decode", req=16, lo=32768, hi=32768, **gqa, page=64, type="bf16", kv="int4",
             spread=8, **none),
        # one request of the longest context of the mixed workload: the length has to be split
        dict(name="decode_one_200k_4bit", kind="decode", req=1, lo=204800, hi=204800, **gqa, page=64, type="bf16", kv="int4",
             spread=9, **none),
        # wide heads, ragged, a window and capped scores over 4-bit pages
        dict(name="decode_wide_4bit", kind="decode", req=61, lo=0, hi=3001, heads=16, kv_heads=2, dim=256, page=32, type="fp16",
             kv="int4", spread=10, **{**none, "window": 700, "cap": 30.0}),
        # one decode step's append into 4-bit pages, and its rows as the cache holds them
        dict(name="append_token_4bit", kind="append", req=16, lo=900, hi=1100, new_lo=1, new_hi=1, **gqa, page=64, type="bf16",
             kv="int4", spread=11, **none),
        # ragged prompts into 4-bit pages, read back as they would be handed to the two-tier cache
        dict(name="append_prompt_4bit", kind="append", req=24, lo=0, hi=700, new_lo=0, new_hi=2000, **gqa, page=32, type="fp16",
             kv="int4", spread=12, **none),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "decode", "decode", "append"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    while kv_heads * group * dim > 8192:
        group = max(1, group // 2)
    heads = kv_heads * group
    case = dict(kind=kind, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128, 256]),
                type=rng.choice(["bf16", "fp16"]), spread=rng.randrange(1 << 20), window=0, cap=0.0, bias=False, prefix=False)
    if kind == "append":
        req = _log(rng, 1, 128)
        case.update(req=req, kv="int4", lo=0, hi=_log(rng, 1, 1000), new_lo=rng.choice([0, 1]),
                    new_hi=_log(rng, 1, max(1, 24000 // req)))
        return case
    case.update(window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), cap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0]),
                bias=rng.random() < 0.3)
    if kind == "attend":
        case["kv"] = rng.choice([case["type"], case["type"], "e4m3", "int4"])
        case["prefix"] = rng.random() < 0.3
        req = _log(rng, 1, 64)
        # requests x tokens x positions x heads within those of the long prompt
        most = (8192 * 8192 * 32) // (req * heads)
        new = _log(rng, 1, max(1, min(8192, int(math.sqrt(most) / 1.5))))
        case.update(req=req, new_lo=rng.choice([0, 1, new]), new_hi=new, lo=0, hi=min(30000, _log(rng, 1, max(1, most // new - new))))
        return case
    # one token: with plain scores over 4-bit pages only
    case["kv"] = rng.choice([case["type"], "e4m3", "int4", "int4"]) if case["cap"] or case["bias"] else "int4"
    req = _log(rng, 1, 128)
    most = (16 * 32768 * 8 * 128) // (req * kv_heads * dim)
    hi = _log(rng, 1, max(2, min(204800, most)))
    case.update(req=req, lo=rng.choice([0, 1, max(1, hi // 4), hi]), hi=hi)
    return case


# ---- sizes that a case stands for ---------------------------------------------------------------

def _lengths(case):
    """Positions each request holds before the call: log-uniform in [lo, hi]; with lo = 0, about one in ten empty."""
    rng = random.Random(1000 + case["spread"])
    lo, hi = case["lo"], case["hi"]
    out = []
    for _ in range(case["req"]):
        empty = lo == 0 and (hi == 0 or rng.random() < 0.1)
        out.append(0 if empty else min(hi, max(lo, _log(rng, max(1, lo), max(1, hi)))))
    return out


def _new_tokens(case):
    """New tokens of each request: uniform in [new_lo, new_hi], and at least one in all."""
    rng = random.Random(2000 + case["spread"])
    out = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["req"])]
    if sum(out) == 0:
        out[-1] = 1
    return out


def _prefixes(case):
    rng = random.Random(3000 + case["spread"])
    most = case["hi"] + case.get("new_hi", 0)
    return [rng.choice([0, 1, rng.randint(0, most)]) if case["prefix"] else 0 for _ in range(case["req"])]


def _cached_bytes(case):
    """Bytes of one row of one head in the pages."""
    d = case["dim"]
    return {"bf16": 2 * d, "fp16": 2 * d, "e4m3": d, "int4": 9 * d // 16}[case["kv"]]


def work(case):
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    row, lengths = _cached_bytes(case), _lengths(case)
    if case["kind"] == "append":
        n = sum(_new_tokens(case))
        # new keys and values, their pages written and read, their values
        return {"bytes": n * 2 * hk * (2 * d + 2 * row + 2 * d), "flops": 4 * n * 2 * hk * d}
    if case["kind"] == "decode":
        seen = sum(min(x, case["window"]) if case["window"] else x for x in lengths)
        return {"bytes": seen * 2 * hk * row + 4 * case["req"] * hq * d, "flops": 4 * seen * hq * d}
    pairs = read = 0
    new = _new_tokens(case)
    for held, n, prefix in zip(lengths, new, _prefixes(case)):
        total, window = held + n, case["window"] or held + n
        pos = torch.arange(held, total, dtype=torch.int64)
        pairs += int((torch.clamp(pos + 1, min=min(prefix, total)) - torch.clamp(pos + 1 - window, min=0)).sum())
        read += total - max(0, held + 1 - window) if n else 0
    return {"bytes": read * 2 * hk * row + 4 * sum(new) * hq * d, "flops": 4 * pairs * hq * d}


# ---- 4-bit rows -----------------------------------------------------------------------------------

def _quantised(x):
    """x [..., d] in 32 bits, under its head's scale -> codes [..., d] and e4m3 scales [..., d / 16]."""
    blocks = x.unflatten(-1, (-1, UNIT))
    seven = torch.full((), 7.0, device=x.device)    # (a number would be taken as its reciprocal: other bits next to a border)
    scale = (blocks.abs().amax(-1) / seven).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    code = torch.where(s > 0, torch.round(blocks / torch.where(s > 0, s, 1.0)).clamp(-7, 7), 0.0) + 8
    return code.flatten(-2).to(torch.uint8), scale


def _pairs(code):
    """codes [..., d] -> bytes [..., d / 2]."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _units(x):
    """x [..., 2, hk, page, d] in 32 bits -> the pages' bytes [..., 2, hk, page / 16, 9 d]."""
    code, scale = _quantised(x.unflatten(-2, (-1, UNIT)))
    scale = scale.view(torch.uint8)
    code = _pairs(code)                                              # [..., 2, hk, units, 16, d / 2]
    k, v = (torch.cat([c.flatten(-2 - extra), s.flatten(-2)], -1) for c, s, extra in (
        (code[..., 0, :, :, :, :], scale[..., 0, :, :, :, :], 0),
        (code[..., 1, :, :, :, :].unflatten(-1, (-1, 16)).transpose(-2, -3), scale[..., 1, :, :, :, :].transpose(-1, -2), 1)))
    return torch.stack([k, v], -4)


def _values(pages, d, dtype=torch.float32):
    """The pages' bytes [..., 2, hk, units, 9 d] -> values [..., 2, hk, page, d] under their heads' scales."""
    code, scale = pages.split([8 * d, d], -1)
    scale = scale.contiguous().view(torch.float8_e4m3fn).to(dtype)
    k, v = code[..., 0, :, :, :], code[..., 1, :, :, :]
    k = k.unflatten(-1, (UNIT, -1))
    v = v.unflatten(-1, (-1, UNIT, 16)).transpose(-2, -3).flatten(-2)
    sk, sv = scale[..., 0, :, :, :].unflatten(-1, (UNIT, -1)), scale[..., 1, :, :, :].unflatten(-1, (-1, UNIT)).transpose(-1, -2)
    byte, s = torch.stack([k, v], -5), torch.stack([sk, sv], -5)     # [..., 2, hk, units, 16, d / 2 and d / 16]
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).to(dtype) - 8
    return (code.unflatten(-1, (-1, UNIT)) * s[..., None]).flatten(-2).flatten(-3, -2)


# ---- inputs -------------------------------------------------------------------------------------

def _slopes(case):
    """2^(-8 (h + 1) / heads): what a score loses per position of distance."""
    h = torch.arange(1, case["heads"] + 1, dtype=torch.float64)
    return (2.0 ** (-8.0 * h / case["heads"])).float().to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt, kv, page = TYPES[case["type"]], TYPES[case["kv"]], case["page"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    four, eight = case["kv"] == "int4", case["kv"] == "e4m3"
    st = {"case": case, "scale": None, "slopes": _slopes(case) if case["bias"] else None}

    held = _lengths(case)
    new = _new_tokens(case) if case["kind"] != "decode" else [0] * case["req"]
    pages_of = [-(-(a + b) // page) for a, b in zip(held, new)]
    n_pages, width = sum(pages_of) + 3, max(1, max(pages_of))
    # pages in no order, as a pool that has been in use hands them out
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((case["req"], width), -1, dtype=torch.int32, device=DEV)
    at = torch.arange(width, device=DEV)
    table[at[None, :] < torch.tensor(pages_of, device=DEV)[:, None]] = order[: sum(pages_of)]
    st["table"] = table
    st["lengths"] = torch.tensor(held, dtype=torch.int32, device=DEV)
    st["next"] = torch.tensor([a + b for a, b in zip(held, new)], dtype=torch.int32, device=DEV)
    shape = (n_pages, 2, hk, page // UNIT, 9 * d) if four else (n_pages, 2, hk, page, d)
    pool = torch.empty(shape, dtype=kv, device=DEV)
    step = max(1, (1 << 27) // (2 * hk * page * d))
    for i in range(0, n_pages, step):
        part = torch.randn(min(step, n_pages - i), 2, hk, page, d, generator=g, device=DEV,
                           dtype=torch.float32 if four or eight else dt)
        if eight:
            part = (part * 110.0).clamp(-E4M3_MAX, E4M3_MAX).to(kv)
        pool[i:i + step] = _units(part) if four else part
    st["pages"] = pool
    if eight:
        st["scale"] = (torch.rand(2, hk, generator=g, device=DEV) * 0.5 + 0.75) / 110.0
    if four:   # powers of two: the scales of the blocks hold the rest
        st["scale"] = 2.0 ** torch.randint(-1, 2, (2, hk), generator=g, device=DEV).float()

    n = sum(new)
    st["offsets"] = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
    if case["kind"] == "append":
        # rows of one projection, some heads and tokens louder than others
        kv_rows = torch.randn(n, 2 * hk * d, generator=g, device=DEV) * torch.rand(n, 1, generator=g, device=DEV).mul(2).exp()
        kv_rows = kv_rows.to(dt)
        st["k"], st["v"] = kv_rows[:, :hk * d].view(n, hk, d), kv_rows[:, hk * d:].view(n, hk, d)
    else:
        # some heads look closely, some broadly
        rows = n if case["kind"] == "attend" else case["req"]
        sharp = torch.rand(1, hq, 1, generator=g, device=DEV) * 3 + 0.5
        st["q"] = (torch.randn(rows, hq, d, generator=g, device=DEV) * sharp).to(dt)
        st["prefix"] = torch.tensor(_prefixes(case), dtype=torch.int32, device=DEV) if case["prefix"] else None
    if case["kind"] == "attend":
        st["most"] = max(new)
    if own:
        from tiered_kv_cache_int8_gb300 import PagedKVCache
        cache = PagedKVCache(n_layers=1, n_pages=n_pages, page_size=page, max_requests=case["req"], max_pages=width,
                             h_q=hq, h_kv=hk, d=d, dtype=dt, kv_dtype="int4" if four else kv, window=case["window"],
                             softcap=case["cap"], slopes=st["slopes"],
                             kv_scale=None if st["scale"] is None else st["scale"][None], pages=pool[None])
        cache.page_table.copy_(table)
        cache.set_lengths(st["lengths"])
        st["cache"] = cache
    return st


# ---- the plain forms ----------------------------------------------------------------------------

def _held(st):
    """Keys and values of every request, [2, r, hk, width * page, d] in 32 bits."""
    case = st["case"]
    held = st["pages"][st["table"].clamp(min=0).long()]
    held = _values(held, case["dim"]) if case["kv"] == "int4" else held.float()
    kv = held.permute(2, 0, 3, 1, 4, 5).flatten(3, 4)
    return kv if st["scale"] is None else kv * st["scale"][:, None, :, None, None]


def _attention(st, q, pos, seen):
    """q [r, t, hq, d] at positions pos [r, t]; seen [r, t, n] -> outputs [r, t, hq, d], lse [r, t, hq]."""
    case = st["case"]
    r, t, hq, d = q.shape
    hk = case["kv_heads"]
    k, v = _held(st)
    g = hq // hk
    rows = q.float().view(r, t, hk, g, d).transpose(1, 2).reshape(r, hk, t * g, d)
    s = torch.matmul(rows, k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(r, hk, t, g, -1)
    if case["cap"]:
        s = s.div_(case["cap"]).tanh_().mul_(case["cap"])
    if case["bias"]:
        far = (pos[:, :, None] - torch.arange(k.shape[2], device=DEV)).abs().float()
        s = s - st["slopes"].view(1, hk, 1, g, 1) * far[:, None, :, None, :]
    s = s.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen.any(1)[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(r, hk, t * g, -1), v).view(r, hk, t, g, d) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + total.log()).squeeze(-1)
    return o.permute(0, 2, 1, 3, 4).reshape(r, t, hq, d).to(q.dtype), lse.permute(0, 2, 1, 3).reshape(r, t, hq)


def _rows_of(st):
    """Each new token's request, its place among the request's, and its position."""
    row = torch.arange(st["k" if "k" in st else "q"].shape[0], device=DEV)
    req = (row[:, None] >= st["offsets"][None, 1:]).sum(1)
    j = row - st["offsets"][req]
    return req, j, st["lengths"][req] + j


def _attend(st):
    case, q = st["case"], st["q"]
    req, j, _ = _rows_of(st)
    r = case["req"]
    padded = torch.zeros(r, st["most"], *q.shape[1:], dtype=q.dtype, device=DEV)
    padded[req, j] = q
    pos = st["lengths"][:, None] + torch.arange(st["most"], device=DEV)
    until = pos + 1 if st["prefix"] is None else torch.maximum(pos + 1, st["prefix"][:, None])
    until = torch.minimum(until, st["next"][:, None])
    at = torch.arange(st["table"].shape[1] * case["page"], device=DEV)
    seen = at < until[:, :, None]
    if case["window"]:
        seen = seen & (at > pos[:, :, None] - case["window"])
    out, lse = _attention(st, padded, pos, seen)
    return out[req, j], lse[req, j]


def _decode(st):
    case = st["case"]
    at = torch.arange(st["table"].shape[1] * case["page"], device=DEV)
    n = st["next"][:, None]
    seen = at < n
    if case["window"]:
        seen = seen & (at >= n - case["window"])
    out, lse = _attention(st, st["q"][:, None], n - 1, seen[:, None])
    return out[:, 0], lse[:, 0]


def _append(st):
    case, pages = st["case"], st["pages"]
    d, hk = case["dim"], case["kv_heads"]
    req, _, pos = _rows_of(st)
    page = st["table"][req, pos // case["page"]].long()
    unit, slot = pos % case["page"] // UNIT, (pos % UNIT).long()
    x = torch.stack([st["k"], st["v"]], 1).float() * (1 / st["scale"])[None, :, :, None]
    code, scale = _quantised(x)                                      # [n, 2, hk, d], [n, 2, hk, d / 16]
    byte = torch.cat([_pairs(code), scale.view(torch.uint8)], -1)    # [n, 2, hk, 9 d / 16]
    e, b = torch.arange(d // 2, device=DEV), torch.arange(d // 16, device=DEV)
    at_k = torch.cat([slot[:, None] * (d // 2) + e, 8 * d + slot[:, None] * (d // 16) + b], 1)
    at_v = torch.cat([(e // 16) * 256 + slot[:, None] * 16 + e % 16, 8 * d + b * UNIT + slot[:, None]], 1)
    at = torch.stack([at_k, at_v], 1)[:, :, None, :]
    where = (page[:, None, None, None], torch.arange(2, device=DEV)[:, None, None], torch.arange(hk, device=DEV)[:, None],
             unit.long()[:, None, None, None], at)
    pages[where] = byte
    # the rows as the pages now hold them
    got = pages[where]
    code = torch.stack([got[..., :d // 2] & 15, got[..., :d // 2] >> 4], -1).flatten(-2).float() - 8
    s = got[..., d // 2:].contiguous().view(torch.float8_e4m3fn).float()
    rows = (code.unflatten(-1, (-1, UNIT)) * s[..., None]).flatten(-2) * st["scale"][None, :, :, None]
    return (st["lengths"] + st["offsets"][1:] - st["offsets"][:-1]).to(torch.int32), rows.to(st["k"].dtype)


def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        cache = st["cache"]
        if kind == "decode":
            return cache.decode(0, st["q"], return_lse=True)
        if kind == "attend":
            return cache.attend(0, st["q"], tok_offsets=st["offsets"], prefix=st["prefix"], return_lse=True)
        cache.append(0, st["k"], st["v"], tok_offsets=st["offsets"])
        return cache.next_lengths, cache.read(0, st["k"].shape[0], tok_offsets=st["offsets"])
    return {"decode": _decode, "attend": _attend, "append": _append}[kind](st)


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _exact_blocks(x):
    """What 4-bit pages hold of x [..., d] (64 bits, under its head's scale)."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    s = torch.clamp(torch.amax(torch.abs(b), dim=-1, keepdim=True) / 7, max=448.0).float().to(torch.float8_e4m3fn).double()
    c = torch.clamp(torch.round(torch.nan_to_num(b / s, nan=0.0, posinf=0.0, neginf=0.0)), -7, 7)
    return (c * s).reshape(x.shape)


def _exact_rows(case, pages, scale, ids):
    """Keys and values [2, hk, n, d] (64 bits) of the pages `ids` of one request."""
    d, held = case["dim"], pages[ids]
    if case["kv"] == "int4":
        parts = []
        for which in (0, 1):
            unit = held[:, which].permute(1, 0, 2, 3).reshape(case["kv_heads"], -1, 9 * d)
            code, s = unit[..., :8 * d], unit[..., 8 * d:].contiguous().view(torch.float8_e4m3fn).double()
            low, high = (code % 16).double() - 8, torch.div(code, 16, rounding_mode="floor").double() - 8
            both = torch.stack((low, high), -1)
            if which == 0:
                x = both.reshape(*unit.shape[:2], 16, d)
                s = s.reshape(*unit.shape[:2], 16, d // 16)
            else:
                x = both.reshape(*unit.shape[:2], d // 32, 16, 32).permute(0, 1, 3, 2, 4).reshape(*unit.shape[:2], 16, d)
                s = s.reshape(*unit.shape[:2], d // 16, 16).permute(0, 1, 3, 2)
            parts.append((x * torch.repeat_interleave(s, 16, dim=-1)).reshape(case["kv_heads"], -1, d))
        kv = torch.stack(parts)
    else:
        kv = held.double().permute(1, 2, 0, 3, 4).flatten(2, 3)
    return kv if scale is None else kv * scale.double()[:, :, None, None]


def exact(case, seed):
    st = prepare(case, seed)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    ends, held, after = st["offsets"].tolist(), st["lengths"].tolist(), st["next"].tolist()
    if case["kind"] == "append":
        x = torch.stack((st["k"], st["v"]), 1).double() / st["scale"].double()[:, :, None]
        return st["next"], _exact_blocks(x) * st["scale"].double()[:, :, None]
    one = case["kind"] == "decode"
    slopes = st["slopes"].double() if case["bias"] else None
    prefixes = _prefixes(case)
    outs, lses = [], []
    for r in range(case["req"]):
        q = (st["q"][r:r + 1] if one else st["q"][ends[r]:ends[r + 1]]).double()
        t, n = q.shape[0], after[r]
        out = torch.zeros(t, hq, d, dtype=torch.float64, device=DEV)
        lse = torch.full((t, hq), -math.inf, dtype=torch.float64, device=DEV)
        outs.append(out)
        lses.append(lse)
        if t == 0 or n == 0:
            continue
        kv = _exact_rows(case, st["pages"], st["scale"], st["table"][r, :-(-n // page)].long())[:, :, :n]
        p = torch.arange(n - t, n, device=DEV)[:, None]
        at = torch.arange(n, device=DEV)[None, :]
        hidden = at > (p if one else torch.clamp(p, min=min(prefixes[r], n) - 1))
        if case["window"]:
            hidden = hidden | (p - at >= case["window"])
        for h in range(hq):
            s = q[:, h] @ kv[0, h * hk // hq].T / math.sqrt(d)
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["bias"]:
                s = s - slopes[h] * (p - at).abs()
            s = s.masked_fill(hidden, -math.inf)
            total = torch.logsumexp(s, -1)
            out[:, h] = torch.exp(s - total[:, None]) @ kv[1, h * hk // hq]
            lse[:, h] = total
    return torch.cat(outs), torch.cat(lses)
