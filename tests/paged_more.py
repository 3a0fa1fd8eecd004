"""Plain 64-bit implementations of prompt attention, of scores with a cap or a distance bias,
and of 4-bit rows, with the tolerances their kernels are held to; and caches to try them on."""
import math

import torch

from tests.paged_plain import HALF_STEP, TINY

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


# ---- 4-bit rows: a byte at a time, as include/hs.h lays them out ---------------------------------

def places(d):
    """Byte of each element's code and of its block's scale in a unit, [2 (keys, values), 16, d]."""
    e = torch.arange(d)
    code, scale = torch.empty(2, 16, d, dtype=torch.long), torch.empty(2, 16, d, dtype=torch.long)
    for i in range(16):
        code[0, i] = i * (d // 2) + e // 2
        scale[0, i] = 8 * d + i * (d // 16) + e // 16
        code[1, i] = (e // 32) * 256 + i * 16 + e % 32 // 2
        scale[1, i] = 8 * d + e // 16 * 16 + i
    return code, scale


def quantise(x, kv_scale):
    """x [n, 2, hk, d] as the kernel takes it (32-bit steps as documented) -> codes (uint8), scale bytes by element."""
    y = x.float() * (1.0 / kv_scale.float())[None, :, :, None]
    b = y.unflatten(-1, (-1, 16))
    top = b.abs().amax(-1, keepdim=True)
    nan = torch.isnan(b).any(-1, keepdim=True)
    # the quotient by 7 rounded to 32 bits, by way of 64 (a quotient of 24-bit numbers is never near a tie of 32 bits there)
    s = (top.double() / torch.full_like(top, 7.0, dtype=torch.float64)).float().clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    s8 = torch.where(nan, torch.full_like(s.view(torch.uint8), 0x7F), s.view(torch.uint8))
    s = s8.view(torch.float8_e4m3fn).float()
    ratio = (b.double() / s.double()).float()
    q = torch.where(s == 0, torch.zeros_like(ratio), torch.round(ratio).clamp(-7, 7))
    code = torch.where(nan, torch.ones_like(q), q + 8)
    return code.nan_to_num(1.0).to(torch.uint8).flatten(-2), s8.expand_as(b).flatten(-2)


def values4(unit_bytes, which, d):
    """Rows [..., 16, d] (64 bits, under the head's scale) of units [..., 9 d]."""
    code_at, scale_at = (t[which].to(unit_bytes.device) for t in places(d))
    c = unit_bytes[..., code_at.flatten()].unflatten(-1, (16, d))
    odd = torch.arange(d, device=unit_bytes.device) % 2 == 1
    c = torch.where(odd, c >> 4, c & 15).double() - 8
    s = unit_bytes[..., scale_at.flatten()].contiguous().view(torch.float8_e4m3fn).unflatten(-1, (16, d)).double()
    return c * s


def put4(pages, page, slot, code, scale):
    """Writes quantised rows (code, scale: [n, 2, hk, d]) at page[n], slot[n] of the bytes [n_pages, 2, hk, units, 9 d]."""
    n, _, hk, d = code.shape
    dev = pages.device
    code_at, scale_at = (t.to(dev) for t in places(d))
    i = (slot % 16).long()
    two = code[..., 0::2] | (code[..., 1::2] << 4)
    which = torch.arange(2, device=dev)[None, :, None, None]
    where = (page.long()[:, None, None, None], which, torch.arange(hk, device=dev)[None, None, :, None],
             (slot // 16).long()[:, None, None, None])
    pages[(*where, code_at[:, i].transpose(0, 1)[:, :, None, 0::2])] = two
    pages[(*where, scale_at[:, i].transpose(0, 1)[:, :, None, 0::16])] = scale[..., 0::16]


# ---- caches ---------------------------------------------------------------------------------------

def rows_of(c, layer, req, n):
    """Keys and values [n, 2, hk, d] of the first n positions of a request as a cache's pages hold them, 64 bits."""
    P = c.page_size
    at = torch.arange(n, device=c.pages.device)
    page = c.page_table[req, at // P].long()
    ok = (page >= 0) & (page < c.n_pages)
    page = torch.where(ok, page, 0)
    pool = c.pages[layer]
    if c.kv_dtype == "int4":
        units = pool[page, :, :, (at % P) // 16]                       # [n, 2, hk, 9 d]
        both = torch.stack([values4(units[:, w], w, c.d) for w in (0, 1)], 1)
        x = both[torch.arange(n, device=at.device), :, :, at % 16]
    else:
        x = pool[page, :, :, at % P].double()
    return (x if c.kv_scale is None else x * c.kv_scale[layer].double()[None, :, :, None]), ok


def make(R, hq, hk, d, page, typ, kv, totals, *, window=0, softcap=0.0, slopes=None, layers=1, layer=0, seed=0, scale=0.0,
         max_requests=None, extra_pages=0, rotary=None, power_of_two=False):
    """A cache with room for `totals` positions of each request, ordinary values in them, NaN everywhere else."""
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    g = torch.Generator(device="cuda").manual_seed(seed + 29)
    counts = [-(-n // page) for n in totals]
    width = max(1, max(counts)) + extra_pages
    n_pages = sum(counts) + R * extra_pages + 2
    quantised = kv in ("e4m3", "int4")
    ks = None
    if quantised:
        ks = (torch.rand(layers, 2, hk, generator=g, device="cuda") + 0.5) / (100 if kv == "e4m3" else 1)
        if power_of_two:
            ks = 2.0 ** torch.randint(-2, 2, (layers, 2, hk), generator=g, device="cuda").float()
    c = PagedKVCache(n_layers=layers, n_pages=n_pages, page_size=page, max_requests=max_requests or R, max_pages=width, h_q=hq,
                     h_kv=hk, d=d, dtype=DT[typ], kv_dtype="int4" if kv == "int4" else DT[kv], window=window, kv_scale=ks,
                     softmax_scale=scale, softcap=softcap, slopes=slopes, rotary=rotary)
    if quantised:
        c.pages.view(torch.uint8).fill_(0x7F)
    else:
        c.pages.fill_(math.nan)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    at = 0
    for r, n in enumerate(totals):
        m = counts[r] + extra_pages
        c.page_table[r, :m] = order[at:at + m]
        at += m
        if n:
            fill(c, layer, r, 0, n, g)
    return c


def fill(c, layer, r, first, n, g):
    """Ordinary values into positions first .. n - 1 of a request."""
    pos = torch.arange(first, n, device="cuda")
    page, slot = c.page_table[r, pos // c.page_size].long(), pos % c.page_size
    x = torch.randn(n - first, 2, c.h_kv, c.d, generator=g, device="cuda")
    if c.kv_dtype == "int4":
        put4(c.pages[layer], page, slot, *quantise(x, c.kv_scale[layer]))
    elif c.kv_dtype == torch.float8_e4m3fn:
        c.pages[layer][page, :, :, slot] = (x * 100).clamp(-448, 448).to(c.kv_dtype)
    else:
        c.pages[layer][page, :, :, slot] = x.to(c.kv_dtype)


# ---- attention --------------------------------------------------------------------------------------

def attend(c, layer, req, q, pos, total, *, prefix=0, scale=None, one=False):
    """q [t, hq, d] at positions pos [t] of a request that holds `total` -> (out, lse, tolerance of out, of lse) in 64 bits.

    one: the tolerance of the one-token attention (weights of 16-bit pages in two parts)."""
    t, hq, d = q.shape
    hk, dev, dtype = c.h_kv, q.device, q.dtype
    scale = scale or 1 / math.sqrt(d)
    out, tol = (torch.zeros(t, hq, d, dtype=torch.float64, device=dev) for _ in range(2))
    lse = torch.full((t, hq), -math.inf, dtype=torch.float64, device=dev)
    tol_lse = torch.zeros(t, hq, dtype=torch.float64, device=dev)
    if total == 0 or t == 0:
        return out, lse, tol, tol_lse
    kv, ok = rows_of(c, layer, req, total)
    at = torch.arange(total, device=dev)
    far = (pos[:, None] - at[None, :]).double()
    seen = (at[None, :] < (pos[:, None] + 1).clamp(min=min(prefix, total))) & ok[None, :]
    if c.cfg.window:
        seen &= far < c.cfg.window
    anyone = seen.any(0)
    kv = torch.where(anyone[:, None, None, None], kv, 0.0)
    slopes = None if c.slopes is None else c.slopes.double()
    quantised = c.kv_scale is not None
    n = seen.sum(1).double()
    for h in range(hq):
        k, v, x = kv[:, 0, h * hk // hq], kv[:, 1, h * hk // hq], q[:, h].double()
        s = x @ k.T * scale
        # a sum of d products in 32 bits (a step each, rounded or cut), the scales
        e = (d + 8) * 2.0 ** -23 * (x.abs() @ k.abs().T * scale) + 2.0 ** -22 * s.abs()
        if quantised:     # queries in 16 bits under a power of two: 2^-25 of their largest
            e = e + 2.0 ** -24 * x.abs().amax(1, keepdim=True) * k.abs().sum(1)[None, :] * scale
        if c.softcap:     # tanh to 2^-20 of itself (a slope of 1 at most), its product
            s = c.softcap * torch.tanh(s / c.softcap)
            e = e + 2.0 ** -19 * s.abs()
        if slopes is not None:
            b = slopes[h] * far.abs()
            s = s - b
            e = e + 2.0 ** -22 * (b.abs() + s.abs())
        s = s.masked_fill(~seen, -math.inf)
        e = torch.where(seen, e, 0.0).amax(1)
        top = torch.logsumexp(s, 1)
        p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top)[:, None])
        out[:, h], lse[:, h] = p @ v, top
        size = p @ v.abs()
        # weights and their sum, sums over n; arguments of the powers of two as differences in 32 bits
        big = torch.where(seen, s.abs(), 0.0).amax(1)
        e_p = 2 * e + 2.0 ** -20 + 2.0 ** -21 * big + (n + 64) * 2.0 ** -23
        # one rounding of each weight to 16 bits (8- and 4-bit pages: fp16), of bf16 and fp16 pages for one token
        # twice; and fp16's smallest spacing under the scale of 2^7
        u_p = HALF_STEP[torch.float16] if quantised else HALF_STEP[dtype] ** (2 if one else 1)
        x = size * (u_p + e_p[:, None]) + 2.0 ** -20 * out[:, h].abs() + n[:, None] * 2.0 ** -32 * v.abs().amax()
        tol[:, h] = x + HALF_STEP[dtype] * (out[:, h].abs() + x) + TINY[dtype]
        tol_lse[:, h] = e + 2.0 ** -20 + 2.0 ** -21 * big + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * top.abs()
    none = ~seen.any(1)
    out[none], tol[none], tol_lse[none] = 0, 0, 0
    return out, lse, tol, tol_lse


def within(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol) & ~((got == want) & torch.isinf(want))      # a NaN is bad
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()} +- {tol[bad][0].item()}")


def slopes_of(hq):
    return (2.0 ** (-8.0 * torch.arange(1, hq + 1, dtype=torch.float64) / hq)).float().cuda()
