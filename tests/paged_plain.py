"""Plain 64-bit implementations of the rotary, paged-append and paged-attention
operators, for the tests, and the tolerances their kernels are held to."""
import math

import torch

# half a step of a rounding to each type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
             torch.float8_e4m3fn: 2.0 ** -4}
# half the spacing of the smallest values
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150,
        torch.float8_e4m3fn: 2.0 ** -10}
E4M3_MAX = 448.0


def frequencies(rot, base=10000.0, scaling=None):
    s = dict(scaling or {})
    kind, factor = s.get("kind"), s.get("factor", 1.0)
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if kind == "linear":
            f /= factor
        elif kind == "by_parts":
            low, high = s.get("low", 1.0), s.get("high", 32.0)
            w = min(1.0, max(0.0, (s["original_context"] * f / (2 * math.pi) - low) / (high - low)))
            f = w * f + (1 - w) * f / factor
        out.append(f)
    return out


def magnitude(scaling=None):
    s = dict(scaling or {})
    return 0.1 * math.log(s["factor"]) + 1.0 if s.get("kind") == "by_parts" and s["factor"] > 1 else 1.0


def rotate(x, pos, freqs, mag=1.0, interleaved=False, sign=1.0):
    """x [n, h, d], pos [n] -> (rotated in 64 bits, bound of the 32-bit computation's error)."""
    y = x.double()
    out, tol = y.clone(), torch.zeros_like(y)
    rot = 2 * len(freqs)
    angle = pos.double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device=x.device)
    c, s = torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]
    ia = torch.arange(rot // 2, device=x.device) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = y[..., ia], y[..., ib]
    out[..., ia] = mag * (a * c - b * s)
    out[..., ib] = mag * (b * c + a * s)
    # per unit of |a| + |b|: the angle as a float in half turns (2^-24 of at most pi), sincospi (2 ulp),
    # its product with the magnitude, the product with a or b, the sum
    unit = math.pi * 2.0 ** -24 + 2 * 2.0 ** -24 + 2.0 ** -24 + 2.0 ** -24 + 2 * 2.0 ** -24
    tol[..., ia] = tol[..., ib] = unit * abs(mag) * (a.abs() + b.abs())
    return out, tol


def stored(x, tol, kv_dtype, scale=None):
    """What a page holds of x [n, h, d] (64 bits), and the bound of its error."""
    if scale is not None:
        x, tol = x / scale[None, :, None], tol / scale[None, :, None] * (1 + 2.0 ** -22) + 2.0 ** -23 * x.abs() / scale[None, :, None]
        x = x.clamp(-E4M3_MAX, E4M3_MAX)
    return x, tol + HALF_STEP[kv_dtype] * (x.abs() + tol) + TINY[kv_dtype]


def attend(q, pages, table_row, length, window, scale, kv_scale=None):
    """One request: q [h_q, d], pages [n_pages, 2, h_kv, P, d] -> (out, lse, tolerance of out, of lse), 64 bits."""
    hq, d = q.shape
    _, _, hk, P, _ = pages.shape
    dev, dtype = q.device, q.dtype
    first = max(0, length - window) if window else 0
    at = torch.arange(first, length, device=dev)
    if length > 0:
        page = table_row[at // P].long()
        ok = (page >= 0) & (page < pages.shape[0])
        at, page = at[ok], page[ok]
    if length == 0 or at.numel() == 0:
        z = torch.zeros(hq, d, dtype=torch.float64, device=dev)
        return z, torch.full((hq,), -math.inf, dtype=torch.float64, device=dev), z, torch.zeros(hq, dtype=torch.float64, device=dev)
    n = at.numel()
    kv = pages[page, :, :, at % P].double()                   # [n, 2, hk, d]
    if kv_scale is not None:
        kv = kv * kv_scale.double()[None, :, :, None]
    k = kv[:, 0].repeat_interleave(hq // hk, dim=1)           # [n, hq, d]
    v = kv[:, 1].repeat_interleave(hq // hk, dim=1)
    q64 = q.double()
    s = torch.einsum("hd,nhd->hn", q64, k) * scale
    lse = torch.logsumexp(s, dim=1)
    p = torch.exp(s - lse[:, None])
    out = torch.einsum("hn,nhd->hd", p, v)
    size = torch.einsum("hn,nhd->hd", p, v.abs())
    # scores: sums of d products in 32 bits (a step each, rounded or cut), the scale, and in 8-bit pages' scale;
    # queries of 8-bit pages in 16 bits under a power of two: 2^-25 of their largest
    dots = torch.einsum("hd,nhd->hn", q64.abs(), k.abs()).amax(1) * scale
    e_s = (d + 8) * 2.0 ** -23 * dots + 2.0 ** -22 * s.abs().amax(1)
    if kv_scale is not None:
        e_s = e_s + 2.0 ** -24 * (q64.abs().amax(1) * k.abs().sum(-1).amax(0)) * scale
    e_p = 2 * e_s + 2.0 ** -20 + (n + 64) * 2.0 ** -23        # weights and their sum, sums over n
    # the weights' rounding: twice to 16 bits (once for 8-bit pages), and fp16's smallest spacing under the
    # scale of 2^7, against a sum that is 1 at least
    u_p = HALF_STEP[torch.float16] if kv_scale is not None else HALF_STEP[dtype] ** 2
    tol = size * (u_p + e_p[:, None]) + 2.0 ** -20 * out.abs() + n * 2.0 ** -32 * v.abs().amax()
    tol = tol + HALF_STEP[dtype] * (out.abs() + tol) + TINY[dtype]
    return out, lse, tol, e_s + 2.0 ** -20 + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * lse.abs()
