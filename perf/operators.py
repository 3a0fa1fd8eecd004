"""Operators measured on one GPU: rotary positions, appending rotated keys and
values to a paged cache, and attention of one new token over that cache.

``run`` computes a case in its plain form (elementary torch operations in 32
bits; angles in 64), or, with ``own`` set, by the calls a user makes of this
package.  ``exact`` gives the same outputs from the definitions in 64 bits.

The paged cache holds, per layer, pages [n_pages, 2, h_kv, page, d]: page p's
keys (index 0) and values (index 1) of ``page`` consecutive positions of one
request.  Position n of request r sits in page table[r, n // page], row n % page.
Eight-bit pages hold value / scale with one scale per kv head for keys and one
for values.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0

# Rotation of every case that rotates: base, and the frequency scaling by its kind.
ROTARY = {"base": 10000.0, "factor": 8.0, "original": 32768, "low": 1.0, "high": 32.0}


def listed():
    gqa = dict(heads=32, kv_heads=8, dim=128)
    return [
        # one decode step of the batch-16 workload: queries and keys of 16 tokens at positions near 32K
        dict(name="rotary_token", kind="rotary", tokens=16, **gqa, rot=128, layout="half", scaling="none",
             far=32768, type="bf16", transpose=False),
        # prompts of a long-context model: half of the head rotated, adjacent pairs, frequencies scaled by parts
        dict(name="rotary_prompt", kind="rotary", tokens=32768, **gqa, rot=64, layout="interleaved",
             scaling="by_parts", far=1048575, type="bf16", transpose=False),
        # the gradients of a rotation in 32 bits, an odd number of tokens
        dict(name="rotary_grad", kind="rotary", tokens=4099, heads=8, kv_heads=1, dim=64, rot=64, layout="half",
             scaling="linear", far=65536, type="fp32", transpose=True),
        # one decode step's append of the batch-16 workload, its queries rotated on the way
        dict(name="append_token", kind="append", req=16, lo=900, hi=1100, new_lo=1, new_hi=1, **gqa, page=64,
             type="bf16", kv="bf16", rot=128, layout="half", scaling="none", spread=1),
        # ragged prompts into 8-bit pages, some requests without a token
        dict(name="append_prompt_8bit", kind="append", req=24, lo=0, hi=700, new_lo=0, new_hi=2000, **gqa, page=32,
             type="bf16", kv="e4m3", rot=128, layout="half", scaling="by_parts", spread=2),
        # a few hundred tokens with wide heads, a quarter of each rotated in adjacent pairs
        dict(name="append_chunk_wide", kind="append", req=5, lo=3, hi=900, new_lo=1, new_hi=333, heads=8, kv_heads=2,
             dim=256, page=16, type="fp16", kv="fp16", rot=64, layout="interleaved", scaling="ntk", spread=3),
        # the one-request 4K workload: latency
        dict(name="decode_tiny_4k", kind="decode", req=1, lo=4096, hi=4096, heads=8, kv_heads=1, dim=128, page=64,
             type="bf16", kv="bf16", window=0, spread=4),
        # the batch-16 workload: 32K positions each
        dict(name="decode_batch16_32k", kind="decode", req=16, lo=32768, hi=32768, **gqa, page=64, type="bf16",
             kv="bf16", window=0, spread=5),
        # one request of the longest context of the mixed workload: the length has to be split
        dict(name="decode_one_200k", kind="decode", req=1, lo=204800, hi=204800, **gqa, page=64, type="bf16",
             kv="bf16", window=0, spread=6),
        # many requests of mixed lengths over 8-bit pages
        dict(name="decode_mixed_8bit", kind="decode", req=64, lo=17, hi=20000, **gqa, page=32, type="bf16",
             kv="e4m3", window=0, spread=7),
        # a sliding window over half-width heads in groups of three, empty requests among them
        dict(name="decode_window", kind="decode", req=33, lo=0, hi=9001, heads=24, kv_heads=8, dim=64, page=16,
             type="fp16", kv="fp16", window=1000, spread=8),
        # a whole step on wide heads: the new token rotated and appended, then attended
        dict(name="step_wide", kind="step", req=64, lo=500, hi=2500, heads=16, kv_heads=2, dim=256, page=64,
             type="bf16", kv="bf16", rot=256, layout="half", scaling="none", window=0, spread=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotary", "append", "decode", "decode", "step"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    while kv_heads * group * dim > 8192:
        group = max(1, group // 2)
    case = dict(kind=kind, heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    if kind != "decode":
        case.update(rot=rng.choice([dim, dim, dim // 2, dim // 4]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "by_parts"]))
    width = (case["heads"] + kv_heads) * dim
    if kind == "rotary":
        case.update(tokens=min(_log(rng, 1, 32768), 32768 * 5120 // width), far=_log(rng, 100, 1048575),
                    type=rng.choice(["bf16", "fp16", "fp32"]), transpose=rng.random() < 0.3)
        return case
    case.update(req=_log(rng, 1, 128), page=rng.choice([16, 32, 64, 128, 256]), type=rng.choice(["bf16", "fp16"]),
                spread=rng.randrange(1 << 20))
    case["kv"] = rng.choice([case["type"], case["type"], "e4m3"])
    if kind == "append":
        case.update(lo=0, hi=_log(rng, 1, 1000))
        most = max(1, 24000 // case["req"])
        case.update(new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, most))
    else:
        # positions x row bytes within those of the batch-16 workload
        most = (16 * 32768 * 8 * 128) // (case["req"] * kv_heads * dim)
        hi = _log(rng, 1, max(2, min(204800, most)))
        lo = rng.choice([0, 1, max(1, hi // 4), hi])
        case.update(lo=lo, hi=hi, window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
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
    """Tokens each request appends: uniform in [new_lo, new_hi], and at least one in all."""
    if case["kind"] == "step":
        return [1] * case["req"]
    rng = random.Random(2000 + case["spread"])
    out = [rng.randint(case["new_lo"], max(case["new_lo"], case["new_hi"])) for _ in range(case["req"])]
    if sum(out) == 0:
        out[-1] = 1
    return out


def work(case):
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    b = BYTES[case["type"]]
    if case["kind"] == "rotary":
        elems = case["tokens"] * (hq + hk) * d
        return {"bytes": 2 * elems * b + 4 * case["tokens"], "flops": 3 * case["tokens"] * (hq + hk) * case["rot"]}
    bk = BYTES[case["kv"]]
    out = {"bytes": 0, "flops": 0}
    lengths = _lengths(case)
    if case["kind"] in ("append", "step"):
        new = _new_tokens(case)
        n = sum(new)
        out["bytes"] += n * d * ((2 * hq + 2 * hk) * b + 2 * hk * bk)
        out["flops"] += 3 * n * (hq + hk) * case["rot"]
        lengths = [x + y for x, y in zip(lengths, new)]
    if case["kind"] in ("decode", "step"):
        seen = sum(min(x, case["window"]) if case["window"] else x for x in lengths)
        out["bytes"] += seen * 2 * hk * d * bk + 2 * case["req"] * hq * d * b
        out["flops"] += 4 * seen * hq * d
    return out


# ---- inputs -------------------------------------------------------------------------------------

def _frequencies(case):
    """Angles per position of each rotated pair, in 64 bits, and the factor on the rotated values.

    pair i of rot / 2:  f_i = base^(-2 i / rot);  linear: f_i / factor;
    ntk: base * factor^(rot / (rot - 2)) in place of base;
    by_parts: w_i f_i + (1 - w_i) f_i / factor with w_i the share of the way that the turns within the original
    context, original * f_i / (2 pi), have gone from `low` to `high`; values times 0.1 ln(factor) + 1."""
    rot, s, factor = case["rot"], case["scaling"], ROTARY["factor"]
    base = ROTARY["base"]
    if s == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    magnitude = 1.0
    if s == "linear":
        f = f / factor
    elif s == "by_parts":
        turns = ROTARY["original"] * f / (2 * math.pi)
        w = ((turns - ROTARY["low"]) / (ROTARY["high"] - ROTARY["low"])).clamp(0, 1)
        f = w * f + (1 - w) * f / factor
        magnitude = 0.1 * math.log(factor) + 1.0
    return f, magnitude


def _plan(case):
    from tiered_kv_cache_int8_gb300 import Rotary
    s = case["scaling"]
    scaling = None
    if s != "none":
        scaling = {"kind": s, "factor": ROTARY["factor"]}
        if s == "by_parts":
            scaling.update(original_context=ROTARY["original"], low=ROTARY["low"], high=ROTARY["high"])
    return Rotary(case["rot"], base=ROTARY["base"], interleaved=case["layout"] == "interleaved", scaling=scaling)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[case["type"]]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32 if dtype.itemsize == 1 else dtype)

    st = {"case": case}
    if case["kind"] == "rotary":
        n = case["tokens"]
        # queries and keys of one projection: rows of a wider tensor
        both = normal(n, (hq + hk) * d)
        st["q"], st["k"] = both[:, :hq * d].view(n, hq, d), both[:, hq * d:].view(n, hk, d)
        st["pos"] = torch.randint(0, case["far"] + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        st["freq"], st["magnitude"] = _frequencies(case)
        st["freq"] = st["freq"].to(DEV)
        if own:
            st["rotary"] = _plan(case)
        return st

    page, kv = case["page"], TYPES[case["kv"]]
    lengths = _lengths(case)
    after = [x + y for x, y in zip(lengths, _new_tokens(case))] if case["kind"] != "decode" else lengths
    pages_of = [-(-n // page) for n in after]
    n_pages, width = sum(pages_of) + 3, max(1, max(pages_of))
    # pages in no order, as a pool that has been in use hands them out
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((case["req"], width), -1, dtype=torch.int32, device=DEV)
    counts = torch.tensor(pages_of, device=DEV)
    held = torch.arange(width, device=DEV)[None, :] < counts[:, None]
    table[held] = order[: sum(pages_of)]
    st["table"] = table
    st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    st["scale"] = None
    pool = torch.empty(n_pages, 2, hk, page, d, dtype=kv, device=DEV)
    step = max(1, (1 << 28) // (2 * hk * page * d))
    for i in range(0, n_pages, step):
        part = normal(min(step, n_pages - i), 2, hk, page, d, dtype=kv)
        if kv.itemsize == 1:   # a little over the largest value in range is met in practice and saturates
            part = (part * 110.0).clamp(-E4M3_MAX, E4M3_MAX).to(kv)
        pool[i:i + step] = part
    st["pages"] = pool
    if kv.itemsize == 1:
        st["scale"] = (torch.rand(2, hk, generator=g, device=DEV) * 0.5 + 0.75) / 110.0
    if case["kind"] in ("append", "step"):
        new = _new_tokens(case)
        n = sum(new)
        qkv = normal(n, (hq + 2 * hk) * d)
        st["q"] = qkv[:, :hq * d].view(n, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hk) * d].view(n, hk, d)
        st["v"] = qkv[:, (hq + hk) * d:].view(n, hk, d)
        ends = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
        st["offsets"] = ends
        st["freq"], st["magnitude"] = _frequencies(case)
        st["freq"] = st["freq"].to(DEV)
    else:
        # some heads look closely, some broadly
        sharp = torch.rand(1, hq, 1, generator=g, device=DEV) * 3 + 0.5
        st["q"] = (torch.randn(case["req"], hq, d, generator=g, device=DEV) * sharp).to(dt)
    if own:
        from tiered_kv_cache_int8_gb300 import PagedKVCache
        cache = PagedKVCache(n_layers=1, n_pages=n_pages, page_size=page, max_requests=case["req"], max_pages=width,
                             h_q=hq, h_kv=hk, d=d, dtype=dt, kv_dtype=kv, window=case.get("window", 0),
                             rotary=_plan(case) if case["kind"] != "decode" else None,
                             kv_scale=None if st["scale"] is None else st["scale"][None], pages=pool[None])
        cache.page_table.copy_(table)
        cache.set_lengths(st["lengths"])
        st["cache"] = cache
    return st


# ---- the plain forms ----------------------------------------------------------------------------

def _rotate(x, pos, freq, magnitude, case, sign=1.0):
    """x [n, h, d] in its type -> rotated in 32 bits."""
    rot = case["rot"]
    angle = pos.double()[:, None] * freq[None, :]
    c, s = (angle.cos() * magnitude).float()[:, None, :], (angle.sin() * (sign * magnitude)).float()[:, None, :]
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    return torch.cat([r, y[..., rot:]], dim=-1)


def _store(x, kv, scale):
    """Values in 32 bits [n, h, d] as the pages hold them."""
    if scale is None:
        return x.to(kv)
    return (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(kv)


def _append(st):
    case, pages = st["case"], st["pages"]
    n = st["k"].shape[0]
    row = torch.arange(n, device=DEV)
    req = (row[:, None] >= st["offsets"][None, 1:]).sum(1)
    pos = st["lengths"][req] + (row - st["offsets"][req])
    page = st["table"][req, pos // case["page"]].long()
    slot = pos % case["page"]
    k = _rotate(st["k"], pos, st["freq"], st["magnitude"], case)
    scale = st["scale"]
    pages[page, 0, :, slot] = _store(k, pages.dtype, None if scale is None else scale[0])
    pages[page, 1, :, slot] = _store(st["v"].float(), pages.dtype, None if scale is None else scale[1])
    q = _rotate(st["q"], pos, st["freq"], st["magnitude"], case).to(st["q"].dtype)
    lengths = st["lengths"] + (st["offsets"][1:] - st["offsets"][:-1])
    return q, lengths.to(torch.int32)


def _decode(st, q, lengths):
    case = st["case"]
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    table = st["table"]
    r, width = table.shape
    held = st["pages"][table.clamp(min=0).long()]                    # [r, width, 2, hk, page, d]
    kv = held.permute(2, 0, 3, 1, 4, 5).reshape(2, r, hk, width * page, d).float()
    if st["scale"] is not None:
        kv = kv * st["scale"][:, None, :, None, None]
    at = torch.arange(width * page, device=DEV)[None, :]
    seen = at < lengths[:, None]
    if case["window"]:
        seen = seen & (at >= lengths[:, None] - case["window"])
    s = torch.matmul(q.float().view(r, hk, hq // hk, d), kv[0].transpose(-1, -2)) / math.sqrt(d)
    s = torch.where(seen[:, None, None, :], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, None, :, None], kv[1], 0.0)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + total.log()).view(r, hq)
    return o.reshape(r, hq, d).to(q.dtype), lse


def run(st):
    case = st["case"]
    kind = case["kind"]
    if own:
        if kind == "rotary":
            return st["rotary"].apply(st["pos"], st["q"], st["k"], transpose=case["transpose"])
        cache = st["cache"]
        if kind == "decode":
            return cache.decode(0, st["q"], return_lse=True)
        q = cache.append(0, st["k"], st["v"], q=st["q"], tok_offsets=st["offsets"])
        if kind == "append":
            return q, st["pages"], cache.next_lengths
        return cache.decode(0, q), st["pages"], cache.next_lengths
    if kind == "rotary":
        sign = -1.0 if case["transpose"] else 1.0
        return tuple(_rotate(x, st["pos"], st["freq"], st["magnitude"], case, sign).to(x.dtype)
                     for x in (st["q"], st["k"]))
    if kind == "decode":
        return _decode(st, st["q"], st["lengths"])
    q, lengths = _append(st)
    if kind == "append":
        return q, st["pages"], lengths
    return _decode(st, q, lengths)[0], st["pages"], lengths


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _turned(case, x, pos, sign=1):
    """Each rotated pair of x (64 bits) as a complex number times magnitude * exp(i angle)."""
    freq, magnitude = _frequencies(case)
    rot = case["rot"]
    turn = torch.polar(torch.full((), magnitude, dtype=torch.float64, device=DEV),
                       sign * torch.outer(pos.double(), freq.to(DEV)))[:, None, :]
    out = x.double().clone()
    if case["layout"] == "half":
        first, second = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        first, second = slice(0, rot, 2), slice(1, rot, 2)
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "rotary":
        sign = -1 if case["transpose"] else 1
        return tuple(_turned(case, st[n], st["pos"], sign) for n in ("q", "k"))
    page, hq, hk = case["page"], case["heads"], case["kv_heads"]
    pages, scale = st["pages"].double(), st["scale"]
    lengths = st["lengths"].tolist()
    q = st["q"].double()
    if kind != "decode":
        ends = st["offsets"].tolist()
        pos = torch.cat([torch.arange(n, n + ends[r + 1] - ends[r], device=DEV) for r, n in enumerate(lengths)])
        k, v, q = _turned(case, st["k"], pos), st["v"].double(), _turned(case, st["q"], pos)
        for r, n in enumerate(lengths):
            rows = slice(ends[r], ends[r + 1])
            at = pos[rows]
            ids, slot = st["table"][r][at // page].long(), at % page
            for which, x in ((0, k[rows]), (1, v[rows])):
                if scale is not None:
                    x = (x / scale[which].double()[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
                pages[ids, which, :, slot] = x
        lengths = [n + ends[r + 1] - ends[r] for r, n in enumerate(lengths)]
        held = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        if kind == "append":
            return q, pages, held
        # what is attended is what the cache and the queries hold: rounded to their types
        stored, pages, q = pages, pages.to(st["pages"].dtype).double(), q.to(st["q"].dtype).double()
    outs, lses = [], []
    for r, n in enumerate(lengths):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            outs.append(torch.zeros(hq, case["dim"], dtype=torch.float64, device=DEV))
            lses.append(torch.full((hq,), -math.inf, dtype=torch.float64, device=DEV))
            continue
        p0 = first // page
        ids = st["table"][r, p0:-(-n // page)].long()
        kv = pages[ids].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, first - p0 * page:n - p0 * page]
        if scale is not None:
            kv = kv * scale.double()[:, :, None, None]
        s = torch.einsum("hgd,hnd->hgn", q[r].view(hk, hq // hk, -1), kv[0]) / math.sqrt(case["dim"])
        lse = torch.logsumexp(s, -1)
        outs.append(torch.einsum("hgn,hnd->hgd", torch.exp(s - lse[..., None]), kv[1]).reshape(hq, -1))
        lses.append(lse.reshape(hq))
    if kind == "decode":
        return torch.stack(outs), torch.stack(lses)
    return torch.stack(outs), stored, held
