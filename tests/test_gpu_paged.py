"""Rotary positions, the paged cache's append and its one-token attention on the GPU,
against plain 64-bit implementations (tests/paged_plain.py, which also derives the
tolerances).  Rows that a call must not use hold NaN or infinities."""
import math

import numpy as np
import pytest

from tests import paged_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tiered_kv_cache_int8_gb300.build import build
    build()
    yield


def T():
    import torch
    return torch


DT = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32", "e4m3": "float8_e4m3fn"}


def dtype(name):
    return getattr(T(), DT[name])


def within(got, want, tol, what):
    torch = T()
    got = got.double()
    bad = ~((got - want).abs() <= tol)       # a NaN is bad
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at "
                           f"{torch.nonzero(bad)[0].tolist()}: {got[bad][0].item()} for {want[bad][0].item()} "
                           f"+- {tol[bad][0].item()}")


# ---- rotary -----------------------------------------------------------------------------------

SCALED = {"none": None, "linear": {"kind": "linear", "factor": 4.0}, "ntk": {"kind": "ntk", "factor": 8.0},
          "parts": {"kind": "by_parts", "factor": 8.0, "original_context": 8192.0}}


@pytest.mark.parametrize("name, n, hq, hk, d, rot, inter, scaling", [
    ("bf16", 16, 32, 8, 128, 128, False, "none"), ("bf16", 1, 1, 1, 64, 64, True, "linear"),
    ("fp16", 77, 8, 2, 256, 64, False, "ntk"), ("fp32", 33, 4, 1, 128, 128, True, "parts"),
    ("fp32", 5, 3, 3, 64, 64, False, "none"), ("bf16", 9000, 2, 1, 64, 32, True, "none"),
    ("bf16", 2500, 5, 1, 128, 64, False, "parts"),
    # sizes that only the one-element kernel takes
    ("bf16", 19, 3, 1, 80, 6, False, "none"), ("fp16", 7, 2, 2, 10, 10, True, "linear"), ("fp32", 11, 1, 1, 2, 2, False, "none"),
    ("bf16", 3, 1, 2, 1024, 1024, False, "none"), ("bf16", 4, 2, 1, 1022, 1022, True, "none"),
])
def test_rotary(name, n, hq, hk, d, rot, inter, scaling):
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    torch.manual_seed(n * d + rot)
    pos = torch.randint(0, 1 << 20, (n,), dtype=torch.int32, device="cuda")
    pos[-1], pos[0] = (1 << 31) - 1, -5
    q, k = (torch.randn(n, h, d, device="cuda").to(dtype(name)) for h in (hq, hk))
    R = Rotary(rot, interleaved=inter, scaling=SCALED[scaling])
    # positions near 2^31 multiply the table's own error: the plain form takes the same frequencies
    freqs = [t / 2.0 ** 64 * 2 * math.pi for t in R.turns]
    far = pos.abs() > 1 << 20
    for transpose in (False, True):
        got = R.apply(pos, q, k, transpose=transpose)
        for x, y in zip((q, k), got):
            want, tol = plain.rotate(x, pos, plain.frequencies(rot, scaling=SCALED[scaling]), plain.magnitude(SCALED[scaling]),
                                     inter, -1.0 if transpose else 1.0)
            exactly, _ = plain.rotate(x, pos, freqs, plain.magnitude(SCALED[scaling]), inter, -1.0 if transpose else 1.0)
            # 2^31 positions times a double's error in the frequency of the plain form
            tol = tol + far[:, None, None] * 2.0 ** 31 * 2.0 ** -50 * 8 * x.double().abs().amax()
            want = torch.where(far[:, None, None], exactly, want)
            tol = tol + plain.HALF_STEP[y.dtype] * (want.abs() + tol) + plain.TINY[y.dtype]
            within(y, want, tol, f"transpose={transpose}")
            assert torch.equal(y[..., rot:], x[..., rot:])
        one = R.apply(pos, k, transpose=transpose)
        assert torch.equal(one, got[1])


@pytest.mark.parametrize("name, shift", [("bf16", 0), ("bf16", 1), ("fp32", 0), ("fp32", 3)])
def test_rotary_strides_and_in_place(name, shift):
    # slices of one projection, [heads][tokens] order, an unaligned start, a broadcast input, in place
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    torch.manual_seed(3)
    n, hq, hk, d = 37, 6, 2, 64
    R = Rotary(d)
    pos = torch.arange(100, 100 + n, dtype=torch.int32, device="cuda")
    wide = torch.randn(n * (hq + 2 * hk) * d + 8, device="cuda").to(dtype(name))[shift:shift + n * (hq + 2 * hk) * d].view(n, -1)
    q, k, v = (wide[:, a * d:b * d].view(n, b - a, d) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    want = R.apply(pos, q.contiguous(), k.contiguous())
    got = R.apply(pos, q, k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ht = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(R.apply(pos, ht), want[0])
    out = torch.full((hq, n, d), 7.0, device="cuda").to(dtype(name)).transpose(0, 1)
    assert R.apply(pos, q, out=out) is out and torch.equal(out, want[0])
    one = q[:1].expand(n, hq, d)
    assert torch.equal(R.apply(pos, one), R.apply(pos, one.contiguous()))
    before = v.clone()
    R.apply(pos, q, k, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)


def test_rotary_gradient():
    # the transposed rotation takes a gradient back: against the formula's and against differences
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    torch.manual_seed(5)
    n, h, d, rot = 13, 3, 64, 48
    R = Rotary(rot, scaling=SCALED["parts"], interleaved=True)
    pos = torch.randint(0, 100000, (n,), dtype=torch.int32, device="cuda")
    x, g = torch.randn(n, h, d, device="cuda"), torch.randn(n, h, d, device="cuda")
    f, mag = plain.frequencies(rot, scaling=SCALED["parts"]), plain.magnitude(SCALED["parts"])
    leaf = x.double().requires_grad_()
    plain.rotate(leaf, pos, f, mag, True)[0].backward(g.double())
    got = R.apply(pos, g, transpose=True)
    _, tol = plain.rotate(g, pos, f, mag, True, -1.0)
    within(got, leaf.grad, tol + 2.0 ** -24 * (leaf.grad.abs() + tol) + 2.0 ** -150, "gradient")
    # linear in x: (f(x + e) - f(x - e)) . g / 2 = e . grad, with each value off by at most its tolerance
    e = torch.randn_like(x)
    up, tu = plain.rotate(x + e, pos, f, mag, True)
    down, td = plain.rotate(x - e, pos, f, mag, True)
    diff = (R.apply(pos, x + e).double() - R.apply(pos, x - e).double()) / 2
    slack = ((tu + td + 2.0 ** -24 * (up.abs() + down.abs() + tu + td)) / 2 * g.double().abs()).sum() + (
        (tol + 2.0 ** -24 * (leaf.grad.abs() + tol)) * e.double().abs()).sum() + (
        2.0 ** -24 * (x.abs() + e.abs()).double() * 2 * mag * (g.double().abs() + g.double().abs().flip(-1))).sum() * 2
    assert abs((diff * g.double()).sum() - (e.double() * got.double()).sum()) <= slack


def test_rotary_refuses_what_the_binding_sees():
    torch = T()
    from tiered_kv_cache_int8_gb300 import HsError, Rotary
    R = Rotary(64)
    x = torch.zeros(4, 2, 64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (pos.long(), pos[:3], pos.cpu()):
        with pytest.raises(ValueError):
            R.apply(bad, x)
    for bad in (x.double(), x[0], x.cpu(), x.transpose(1, 2)):
        with pytest.raises(ValueError):
            R.apply(pos, bad)
    with pytest.raises(ValueError):
        R.apply(pos, x, out=x[:2])
    with pytest.raises(ValueError):
        R.apply(pos, x, x.half())
    with pytest.raises(HsError):
        R.apply(pos, x[..., :32].contiguous())        # rot_dim above d
    with pytest.raises(HsError):
        R.apply(pos, x, out=x[:1].expand(4, 2, 64))   # outputs share memory
    for bad in (dict(scaling={"kind": "no"}), dict(scaling={"kind": "linear"}), dict(scaling={"kind": "linear", "factor": 2, "low": 1}),
                dict(inv_freq=[1.0]), dict(magnitude=0.0), dict(inv_freq=[1.0] * 32, scaling={"kind": "linear", "factor": 2})):
        with pytest.raises(ValueError):
            Rotary(64, **bad)
    with pytest.raises(HsError):
        Rotary(63)
    assert R.apply(pos[:0], x[:0]).shape == (0, 2, 64)


# ---- the paged cache --------------------------------------------------------------------------

def filled(shape, dt, g, poison):
    """A pool of ordinary values, or of NaN (8-bit pages: of NaN bytes)."""
    torch = T()
    if poison:
        if dt == torch.float8_e4m3fn:
            return torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(dt)
        return torch.full(shape, math.nan, dtype=dt, device="cuda")
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * 100).clamp(-448, 448).to(dt) if dt == torch.float8_e4m3fn else x.to(dt)


def make(R, hq, hk, d, page, typ, kv, lengths, window=0, rotary=None, layers=1, layer=0, spare=2, seed=0, extra_pages=0, scale=0.0,
         max_requests=None):
    """A cache whose requests hold `lengths` positions of ordinary values, everything else NaN."""
    torch = T()
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    g = torch.Generator(device="cuda").manual_seed(seed + 17)
    counts = [-(-n // page) for n in lengths]
    width = max(1, max(counts)) + extra_pages
    n_pages = sum(counts) + R * extra_pages + spare
    dt, kt = dtype(typ), dtype(kv)
    ks = (torch.rand(layers, 2, hk, generator=g, device="cuda") + 0.5) / 100 if kv == "e4m3" else None
    c = PagedKVCache(n_layers=layers, n_pages=n_pages, page_size=page, max_requests=max_requests or R, max_pages=width, h_q=hq,
                     h_kv=hk, d=d, dtype=dt, kv_dtype=kt, window=window, rotary=rotary, kv_scale=ks, softmax_scale=scale)
    c.pages.copy_(filled(c.pages.shape, kt, g, True))
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    at = 0
    for r, n in enumerate(lengths):
        m = counts[r] + extra_pages
        c.page_table[r, :m] = order[at:at + m]
        at += m
        if n:
            pos = torch.arange(n, device="cuda")
            rows = filled((n, 2, hk, d), kt, g, False)
            raw = c.pages[layer].view(torch.uint8) if kv == "e4m3" else c.pages[layer]
            rows = rows.view(torch.uint8) if kv == "e4m3" else rows
            raw[c.page_table[r][pos // page].long(), :, :, pos % page] = rows
    c.set_lengths(torch.tensor(list(lengths) + [0] * ((max_requests or R) - R), dtype=torch.int32, device="cuda"))
    return c, g


def check_decode(c, q, lengths, layer=0, window=0, scale=None, ids=None, out=None, lse=None):
    torch = T()
    if out is None:
        out, lse = c.decode(layer, q, return_lse=True, req_ids=None if ids is None else
                            torch.tensor(ids, dtype=torch.int32, device="cuda"))
    pages = c.pages[layer]
    for i in range(q.shape[0]):
        r = i if ids is None else ids[i]
        want, wl, tol, tl = plain.attend(q[i], pages, c.page_table[r], lengths[r], window, scale or 1 / math.sqrt(c.d),
                                         None if c.kv_scale is None else c.kv_scale[layer])
        within(out[i], want, tol, f"out of request {r} (length {lengths[r]})")
        if lengths[r] == 0:
            assert (lse[i] == -math.inf).all()
        else:
            within(lse[i], wl, tl, f"lse of request {r} (length {lengths[r]})")
    return out, lse


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 130, 1000]


@pytest.mark.parametrize("typ, kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq, hk, page", [(4, 4, 16), (8, 1, 64), (12, 4, 32), (32, 2, 128), (40, 1, 256), (7, 1, 16)])
def test_decode_lengths_and_heads(typ, kv, d, hq, hk, page):
    torch = T()
    c, g = make(len(LENGTHS), hq, hk, d, page, typ, kv, LENGTHS, seed=hq * d + page)
    q = (torch.randn(len(LENGTHS), hq, d, generator=g, device="cuda") * 2).to(dtype(typ))
    check_decode(c, q, LENGTHS)
    assert c.device_error() == 0


@pytest.mark.parametrize("typ, kv", [("bf16", "bf16"), ("fp16", "e4m3")])
@pytest.mark.parametrize("window", [1, 5, 16, 100, 999, 5000])
def test_decode_window(typ, kv, window):
    torch = T()
    lengths = [0, 1, 4, 16, 17, 100, 101, 999, 1000, 1001, 3000]
    c, g = make(len(lengths), 8, 2, 128, 32, typ, kv, lengths, window=window)
    q = torch.randn(len(lengths), 8, 128, generator=g, device="cuda").to(dtype(typ))
    # positions before the window are not used, whatever they hold
    for r, n in enumerate(lengths):
        for pos in range(max(0, n - window) // 32 * 32, max(0, n - window)):
            if kv == "e4m3":
                c.pages.view(torch.uint8)[0, c.page_table[r, pos // 32].long(), :, :, pos % 32] = 0x7F
            else:
                c.pages[0, c.page_table[r, pos // 32].long(), :, :, pos % 32] = math.nan
    check_decode(c, q, lengths, window=window)


@pytest.mark.parametrize("lengths", [[70000], [40001, 3], [5000] * 3, [1] * 300, list(range(200)), [0] * 5, [2049] * 64])
@pytest.mark.parametrize("typ, kv, hq, hk, d", [("bf16", "bf16", 32, 8, 128), ("fp16", "e4m3", 8, 1, 64)])
def test_decode_splits(lengths, typ, kv, hq, hk, d):
    # long and few, short and many: the work is cut across requests and heads and joined
    torch = T()
    c, g = make(len(lengths), hq, hk, d, 64, typ, kv, lengths, seed=len(lengths))
    q = torch.randn(len(lengths), hq, d, generator=g, device="cuda").to(dtype(typ))
    out, lse = check_decode(c, q, lengths)
    again, lse2 = c.decode(0, q, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)      # the same bits from call to call


@pytest.mark.parametrize("typ, kv, hq, hk, d, page", [("bf16", "bf16", 32, 8, 128, 64), ("fp16", "e4m3", 40, 2, 64, 16),
                                                      ("bf16", "e4m3", 8, 8, 256, 32), ("fp16", "fp16", 12, 4, 256, 128)])
@pytest.mark.parametrize("most", [40, 512, 513, 1024, 1025])
def test_decode_short_contexts(typ, kv, hq, hk, d, page, most):
    # tables whose width decides between whole segments for each CTA and shared ones
    torch = T()
    for R in (1, 9, 40):
        lengths = [(most if r == 0 else (97 * r + most // 3) % (most + 1)) for r in range(R)]
        if R > 2:
            lengths[2] = 0
        c, g = make(R, hq, hk, d, page, typ, kv, lengths, seed=R + most)
        q = torch.randn(R, hq, d, generator=g, device="cuda").to(dtype(typ))
        check_decode(c, q, lengths)
        assert c.device_error() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_values_at_the_border(kv):
    # large and tiny scores, a row that wins alone, equal rows, zero queries
    torch = T()
    lengths = [500, 500, 500, 500, 33]
    c, g = make(5, 4, 1, 128, 64, "bf16", kv, lengths)
    q = torch.randn(5, 4, 128, generator=g, device="cuda")
    q[0] *= 30
    q[1] *= 1e-30
    q[2] = 0
    q[3] *= 1e4
    q = q.to(torch.bfloat16)
    check_decode(c, q, lengths)
    # all scores far below zero: the maximum is taken out
    with torch.no_grad():
        k = c.pages[0].view(torch.uint8) if kv == "e4m3" else c.pages[0]
        pos = torch.arange(33, device="cuda")
        one = torch.full((128,), -3.0, device="cuda").to(c.kv_dtype)
        k[c.page_table[4][pos // 64].long(), 0, 0, pos % 64] = one.view(torch.uint8) if kv == "e4m3" else one
        q[4] = 40.0
    out, lse = check_decode(c, q, lengths)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_decode_ids_scale_strides_and_layers():
    torch = T()
    lengths = [40, 0, 333, 64, 1, 129]
    c, g = make(6, 12, 4, 128, 16, "fp16", "fp16", lengths, layers=3, layer=2, scale=0.3)
    wide = torch.randn(4, 14 * 128, generator=g, device="cuda").half()
    q = wide[:, 128:13 * 128].view(4, 12, 128)
    ids = [5, 2, 1, 0]
    check_decode(c, q, lengths, layer=2, scale=0.3, ids=ids)
    ht = torch.randn(12, 4, 128, generator=g, device="cuda").half().transpose(0, 1)
    check_decode(c, ht, lengths, layer=2, scale=0.3, ids=ids)
    # lengths of the caller's, and an output of the caller's
    other = torch.tensor([40, 0, 100, 1, 1, 17], dtype=torch.int32, device="cuda")
    out = torch.full((4, 12, 128), 9.0, device="cuda").half()
    got, lse = c.decode(2, ht, lengths=other, out=out, return_lse=True, req_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
    assert got is out
    check_decode(c, ht, other.tolist(), layer=2, scale=0.3, ids=ids, out=out, lse=lse)
    assert c.device_error() == 0


def test_decode_skips_bad_requests_and_pages():
    torch = T()
    from tiered_kv_cache_int8_gb300 import hs
    lengths = [100, 200, 64, 40]
    c, g = make(4, 4, 1, 128, 32, "bf16", "bf16", lengths, max_requests=5)
    q = torch.randn(5, 4, 128, generator=g, device="cuda").bfloat16()
    ids = torch.tensor([0, 7, 2, -1, 3], dtype=torch.int32, device="cuda")
    out, lse = c.decode(0, q, req_ids=ids, return_lse=True)
    assert c.device_error() == hs.HS_DEVERR_REQ_RANGE
    assert (out[[1, 3]] == 0).all() and (lse[[1, 3]] == -math.inf).all()
    check_decode(c, q[[0, 2, 4]].contiguous(), lengths, ids=[0, 2, 3], out=out[[0, 2, 4]], lse=lse[[0, 2, 4]])
    # lengths outside the table
    bad = torch.tensor([-3, 200, c.max_pages * 32 + 1, 40, 0], dtype=torch.int32, device="cuda")
    out, lse = c.decode(0, q[:4], lengths=bad, return_lse=True)
    assert c.device_error() == hs.HS_DEVERR_REQ_RANGE | hs.HS_DEVERR_CAPACITY
    assert (out[[0, 2]] == 0).all() and (lse[[0, 2]] == -math.inf).all()
    # pages that are out of range leave their positions out
    c.page_table[1, 2] = c.n_pages
    c.page_table[1, 4] = -7
    c.page_table[3] = -1
    out, lse = c.decode(0, q[:4], return_lse=True)
    assert c.device_error() & hs.HS_DEVERR_PAGE
    check_decode(c, q[:2].contiguous(), lengths, out=out[:2], lse=lse[:2])
    assert (out[3] == 0).all() and (lse[3] == -math.inf).all()


def test_decode_far_pages():
    # pages beyond 2^31 elements and 4 GiB of the pool, several requests on the same pages
    torch = T()
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    n_pages, page, hk, d = 20000, 256, 2, 128
    c = PagedKVCache(n_layers=1, n_pages=n_pages, page_size=page, max_requests=3, max_pages=4, h_q=4, h_kv=hk, d=d)
    far = [n_pages - 1, n_pages - 7, 17001, 1]
    g = torch.Generator(device="cuda").manual_seed(1)
    for p in far:
        c.pages[0, p] = torch.randn(2, hk, page, d, generator=g, device="cuda").bfloat16()
    for r in range(3):
        c.page_table[r] = torch.tensor(far, dtype=torch.int32)
    lengths = [1024, 700, 3]
    c.set_lengths(torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    q = torch.randn(3, 4, d, generator=g, device="cuda").bfloat16()
    check_decode(c, q, lengths)
    k = torch.randn(2, hk, d, generator=g, device="cuda").bfloat16()
    c.set_lengths(torch.tensor([600, 100, 10], dtype=torch.int32, device="cuda"))
    c.append(0, k, k * 2, req_ids=torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(c.pages[0, 17001, 0, :, 600 % 256], k[0]) and torch.equal(c.pages[0, far[0], 1, :, 100], k[1] * 2)


# ---- append -----------------------------------------------------------------------------------

def expected_append(c, layer, k, v, offs, ids, lengths, freqs, mag, inter):
    """{(page, which, slot): (values, tolerance)} of every stored row, 64 bits, and each row's position."""
    torch = T()
    rows, pos = {}, {}
    for i, r in enumerate(ids):
        for j, t in enumerate(range(offs[i], offs[i + 1])):
            pos[t] = lengths[r] + j
    P = c.page_size
    if not pos:
        return rows, pos
    ts = sorted(pos)
    at = torch.tensor([pos[t] for t in ts], device="cuda")
    kk, kt = plain.rotate(k[ts], at, freqs, mag, inter) if freqs else (k[ts].double(), torch.zeros_like(k[ts].double()))
    vv = v[ts].double()
    for which, (x, tol) in enumerate(((kk, kt), (vv, torch.zeros_like(vv)))):
        x, tol = plain.stored(x, tol, c.kv_dtype, None if c.kv_scale is None else c.kv_scale[layer, which].double())
        who = {t: r for i, r in enumerate(ids) for t in range(offs[i], offs[i + 1])}
        for n, t in enumerate(ts):
            rows[int(c.page_table[who[t], pos[t] // P]), which, pos[t] % P] = (x[n], tol[n])
    return rows, pos


@pytest.mark.parametrize("typ, kv, d, hq, hk, page, rot, inter, scaling", [
    ("bf16", "bf16", 128, 32, 8, 64, 128, False, "none"), ("fp16", "fp16", 256, 4, 2, 16, 64, True, "ntk"),
    ("bf16", "e4m3", 128, 8, 4, 32, 128, False, "parts"), ("fp16", "e4m3", 64, 6, 3, 256, 32, True, "linear"),
    ("bf16", "bf16", 64, 5, 1, 128, 2, False, "none"), ("fp16", "fp16", 64, 2, 2, 32, 6, True, "none"),
    ("bf16", "e4m3", 64, 4, 2, 16, 4, False, "none"), ("bf16", "bf16", 128, 8, 2, 16, 0, False, "none"),
])
@pytest.mark.parametrize("ragged", [False, True])
def test_append(typ, kv, d, hq, hk, page, rot, inter, scaling, ragged):
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    lengths = [0, 1, page - 1, page, 3 * page + 5, 100, 0]
    rotary = Rotary(rot, interleaved=inter, scaling=SCALED[scaling]) if rot else None
    c, g = make(7, hq, hk, d, page, typ, kv, lengths, rotary=rotary, layers=2, layer=1, extra_pages=4, seed=d + page)
    ids = [4, 0, 2, 6, 1]
    counts = [3, 0, page + 2, 1, 2 * page] if ragged else [4] * 5
    offs = [2 + sum(counts[:i]) for i in range(6)] if ragged else [4 * i for i in range(6)]
    n = offs[-1] + (3 if ragged else 0)          # rows before and behind belong to nobody
    dt = dtype(typ)
    qkv = torch.randn(n, (hq + 2 * hk) * d, generator=g, device="cuda").to(dt)
    q, k, v = qkv[:, :hq * d].view(n, hq, d), qkv[:, hq * d:(hq + hk) * d].view(n, hk, d), qkv[:, (hq + hk) * d:].view(n, hk, d)
    if kv == "e4m3":
        v[offs[0], 0, 0], v[offs[0], 0, 1], v[offs[0], 0, 2] = 1e4, -1e4, -0.0    # saturates
    if ragged:
        qkv[:2] = math.nan
        qkv[offs[-1]:] = math.nan
    before = c.pages.clone()
    q_out = torch.full((n, hq, d), 5.0, device="cuda").to(dt)
    raw = c.pages.view(torch.uint8) if kv == "e4m3" else c.pages
    freqs = plain.frequencies(rot, scaling=SCALED[scaling]) if rot else None
    mag = plain.magnitude(SCALED[scaling])
    kw = dict(q=q, q_out=q_out) if rot else {}
    got = c.append(1, k, v, req_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"),
                   tok_offsets=torch.tensor(offs, dtype=torch.int32, device="cuda") if ragged else None, **kw)
    rows, pos = expected_append(c, 1, k, v, offs, ids, lengths, freqs, mag, inter)
    raw_before = before.view(torch.uint8) if kv == "e4m3" else before
    mask = torch.ones(raw.shape[1:], dtype=torch.bool, device="cuda")
    for (p, which, slot), (want, tol) in rows.items():
        within(c.pages[1, p, which, :, slot].float(), want, tol, f"row {p} {which} {slot}")
        mask[p, which, :, slot] = False
    same = raw.view(torch.uint8) == raw_before.view(torch.uint8)         # bits: the pool holds NaN
    es = raw.element_size()
    assert same[0].all() and (same[1] | ~mask.repeat_interleave(es, dim=-1)).all(), "a row outside the call changed"
    if rot:
        assert got is q_out
        at = torch.tensor([pos.get(t, 0) for t in range(n)], device="cuda")
        mine = torch.tensor([t in pos for t in range(n)], device="cuda")
        want, tol = plain.rotate(torch.nan_to_num(q), at, freqs, mag, inter)
        tol = tol + plain.HALF_STEP[dt] * (want.abs() + tol) + plain.TINY[dt]
        within(q_out[mine], want[mine], tol[mine], "q")
        assert (q_out[~mine] == 5.0).all()
    want = list(lengths)
    for i, r in enumerate(ids):
        want[r] += offs[i + 1] - offs[i]
    assert c.next_lengths.tolist() == want and c.lengths.tolist() == lengths
    assert c.device_error() == 0


@pytest.mark.parametrize("R", [1, 31, 32, 33, 65])
def test_append_counts_of_requests(R):
    # up to 32 requests are found another way than more
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary, hs
    counts = [(3 * r + 1) % 4 for r in range(R)]
    counts[-1] += 2
    lengths = [(5 * r) % 40 for r in range(R)]
    offs = [1 + sum(counts[:i]) for i in range(R + 1)]
    ids = [(7 * r + 3) % R for r in range(R)] if R % 7 else list(range(R))
    assert sorted(ids) == list(range(R))
    c, g = make(R, 4, 2, 64, 16, "bf16", "bf16", lengths, rotary=Rotary(32), extra_pages=1)
    n = offs[-1] + 2
    q, k, v = (torch.randn(n, h, 64, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    qo = torch.full_like(q, 5.0)
    c.append(0, k, v, q=q, q_out=qo, req_ids=i32(ids), tok_offsets=i32(offs))
    rows, pos = expected_append(c, 0, k, v, offs, ids, lengths, plain.frequencies(32), 1.0, False)
    assert len(rows) == 2 * sum(counts)
    for (p, which, slot), (want, tol) in rows.items():
        within(c.pages[0, p, which, :, slot], want, tol, f"row {p} {which} {slot}")
    ts = sorted(pos)
    want, tol = plain.rotate(q[ts], torch.tensor([pos[t] for t in ts], device="cuda"), plain.frequencies(32))
    within(qo[ts], want, tol + 2.0 ** -8 * (want.abs() + tol) + plain.TINY[q.dtype], "q")
    others = [t for t in range(n) if t not in pos]
    assert (qo[others] == 5.0).all()
    want = list(lengths)
    for i, r in enumerate(ids):
        want[r] += counts[i]
    assert c.next_lengths.tolist() == want and c.device_error() == 0
    # a bad id among them: only its request is skipped
    if R > 1:
        b = c.pages.view(torch.int16).clone()
        bad = list(ids)
        bad[R // 2] = R
        c.append(0, k * 2, v * 2, req_ids=i32(bad), tok_offsets=i32(offs))
        assert c.device_error() == hs.HS_DEVERR_REQ_RANGE
        i, r = R // 2, ids[R // 2]
        for j in range(counts[i]):
            at = lengths[r] + j
            assert torch.equal(c.pages.view(torch.int16)[0, c.page_table[r, at // 16].long(), :, :, at % 16],
                               b[0, c.page_table[r, at // 16].long(), :, :, at % 16])


def test_append_many_requests_and_long_prompts():
    # the search over many offsets (most of them empty), and CTAs that take several tokens
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    R, hk, d, page = 2500, 1, 64, 16
    counts = [(7 * r) % 5 if r % 3 else 0 for r in range(R)]
    counts[1234] = 900
    lengths = [r % 9 for r in range(R)]
    c, g = make(R, 1, hk, d, page, "bf16", "bf16", [0] * R, rotary=Rotary(d), extra_pages=58)
    c.set_lengths(torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    offs = np.concatenate([[0], np.cumsum(counts)])
    n = int(offs[-1])
    k = torch.randn(n, hk, d, generator=g, device="cuda").bfloat16()
    c.append(0, k, k, tok_offsets=torch.tensor(offs, dtype=torch.int32, device="cuda"))
    who = torch.tensor(np.repeat(np.arange(R), counts), device="cuda")
    pos = torch.tensor(np.concatenate([np.arange(lengths[r], lengths[r] + m) for r, m in enumerate(counts)]), device="cuda")
    page_of = c.page_table[who, pos // page].long()
    assert torch.equal(c.pages[0][page_of, 1, :, pos % page], k)
    want, tol = plain.rotate(k, pos, plain.frequencies(d))
    within(c.pages[0][page_of, 0, :, pos % page], want, tol + 2.0 ** -8 * (want.abs() + tol) + plain.TINY[k.dtype], "keys")
    assert torch.equal(c.next_lengths, c.lengths + torch.tensor(counts, device="cuda"))
    written = torch.zeros(c.n_pages, page, dtype=torch.bool, device="cuda")
    written[page_of, pos % page] = True
    assert torch.isnan(c.pages[0][:, 0, 0, :, 0][~written]).all()


def test_append_skips_bad_requests_pages_and_offsets():
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary, hs
    dev = "cuda"

    def fresh():
        return make(4, 2, 1, 64, 16, "bf16", "bf16", [3, 16, 30, 5], rotary=Rotary(64), spare=1)

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    c, g = fresh()
    k = torch.randn(8, 1, 64, generator=g, device=dev).bfloat16()
    q = torch.randn(8, 2, 64, generator=g, device=dev).bfloat16()
    qo = torch.full_like(q, 5.0)
    bits = lambda: c.pages.view(torch.int16).clone()   # noqa: E731
    # ids out of range
    b = bits()
    c.append(0, k[:2], k[:2], q=q[:2], q_out=qo[:2], req_ids=i32(4, -1))
    assert c.device_error() == hs.HS_DEVERR_REQ_RANGE and torch.equal(bits(), b) and (qo == 5.0).all()
    # tokens past the table (2 pages of 16 each): request 2 is skipped whole, request 0 is not
    c, g = fresh()
    c.append(0, k[:6], k[:6], q=q[:6], q_out=qo[:6], req_ids=i32(2, 0))
    assert c.device_error() == hs.HS_DEVERR_CAPACITY
    assert c.next_lengths.tolist() == [6, 16, 30, 5] and (qo[:3] == 5.0).all() and (qo[3:6] != 5.0).any()
    assert torch.equal(c.pages[0, c.page_table[0, 0].long(), 1, 0, 3:6], k[3:6, 0])
    # a negative length
    c, g = fresh()
    c.set_lengths(i32(-1, 16, 30, 5))
    c.append(0, k[:1], k[:1], req_ids=i32(0))
    assert c.device_error() == hs.HS_DEVERR_CAPACITY
    # a page id out of range: its positions are not stored, the others are
    c, g = fresh()
    c.page_table[1, 1] = c.n_pages
    b = bits()
    c.append(0, k[:1], k[:1], req_ids=i32(1))
    assert c.device_error() == hs.HS_DEVERR_PAGE and torch.equal(bits(), b) and c.next_lengths.tolist() == [3, 17, 30, 5]
    # offsets that decrease or leave the rows
    for offs in ((0, 2, 1, 3), (-2, 0, 1, 2), (0, 1, 2, 9)):
        c, g = fresh()
        c.append(0, k[:4], k[:4], tok_offsets=i32(*offs))
        assert c.device_error() & hs.HS_DEVERR_OFFSETS


# ---- together, and as a program uses them -------------------------------------------------------

def steps(c, inputs, layers, run):
    """`run` one step per entry: append and attend in every layer, then commit."""
    outs = []
    for step in inputs:
        outs.append([run(c, l, *step[l]) for l in range(layers)])
        c.commit()
    return outs


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_steps_of_a_model(kv):
    # prompts of different lengths, then single tokens, over two layers, pages handed out on the way
    torch = T()
    from tiered_kv_cache_int8_gb300 import PagedKVCache, Rotary
    g = torch.Generator(device="cuda").manual_seed(4)
    L, R, hq, hk, d, page = 2, 3, 8, 2, 128, 16
    scale = torch.full((L, 2, hk), 0.02, device="cuda") if kv == "e4m3" else None
    rot = Rotary(64, base=500000.0)
    freqs = plain.frequencies(64, 500000.0)
    c = PagedKVCache(n_layers=L, n_pages=40, page_size=page, max_requests=R, max_pages=8, h_q=hq, h_kv=hk, d=d,
                     kv_dtype=dtype(kv), rotary=rot, kv_scale=scale)
    c.pages.copy_(filled(c.pages.shape, c.kv_dtype, g, True))
    prompts = [19, 1, 40]
    held = [0, 0, 0]
    offs = torch.tensor([0, 19, 20, 60], dtype=torch.int32, device="cuda")
    for step in range(7):
        new = prompts if step == 0 else [1, 1, 1]
        n = sum(new)
        for r in range(R):
            c.reserve(r, held[r] + new[r])
        last = torch.tensor(np.cumsum(new) - 1, device="cuda")
        for l in range(L):
            q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for h in (hq, hk, hk))
            qr = c.append(l, k, v, q=q, tok_offsets=offs if step == 0 else None)
            rows, pos = expected_append(c, l, k, v, [0] + np.cumsum(new).tolist(), range(R), held, freqs, 1.0, False)
            for (p, which, slot), (want, tol) in rows.items():
                within(c.pages[l, p, which, :, slot].float(), want, tol, "stored row")
            check_decode(c, qr[last].contiguous(), [h + m for h, m in zip(held, new)], layer=l)
        held = [h + m for h, m in zip(held, new)]
        c.commit()
        assert c.lengths.tolist() == held
    assert c.device_error() == 0
    free = c.free_pages()
    c.release(2)
    assert c.free_pages() == free + 3 and c.lengths.tolist() == held[:2] + [0] and (c.page_table[2] == -1).all()
    with pytest.raises(MemoryError):
        for r in range(R):
            c2 = PagedKVCache(n_layers=1, n_pages=2, page_size=16, max_requests=R, max_pages=8, h_q=hq, h_kv=hk, d=d)
            c2.reserve(0, 33)
    with pytest.raises(ValueError):
        c.reserve(0, 8 * 16 + 1)


def small_step(seed=0, kv="bf16"):
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    lengths = [700, 33, 0, 2000]
    c, g = make(4, 8, 2, 128, 32, "bf16", kv, lengths, rotary=Rotary(128), extra_pages=1, seed=seed)
    q, k, v = (torch.randn(4, h, 128, generator=g, device="cuda").bfloat16() for h in (8, 2, 2))
    return c, q, k, v, [n + 1 for n in lengths]


def test_captured_steps_share_nothing():
    # two graphs of the same cache, replayed after new inputs came, on two streams at once
    torch = T()
    c, q, k, v, after = small_step()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    c.append(0, k, v, q=q)
    c.decode(0, q)
    torch.cuda.synchronize()
    graphs, ins, outs = [], [], []
    for s in streams:
        gr, qi = torch.cuda.CUDAGraph(), torch.zeros_like(q)
        with torch.cuda.graph(gr, stream=s):
            o = c.decode(0, qi, return_lse=True)
        graphs.append(gr), ins.append(qi), outs.append(o)
    for rep in range(20):
        qs = [torch.randn_like(q) for _ in graphs]
        for qi, new in zip(ins, qs):
            qi.copy_(new)
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for (o, l), new in zip(outs, qs):
            check_decode(c, new, after, out=o, lse=l)
    # a captured step that appends: replayed, it stores what its inputs then hold
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        qr = c.append(0, k, v, q=q)
        o, l = c.decode(0, qr, return_lse=True)
        c.commit()
    for _ in range(3):
        before = c.lengths.tolist()
        for x in (q, k, v):
            x.copy_(torch.randn_like(x))
        gr.replay()
        torch.cuda.synchronize()
        after = [n + 1 for n in before]
        assert c.lengths.tolist() == after
        for r, n in enumerate(before):
            assert torch.equal(c.pages[0, c.page_table[r, n // 32].long(), 1, :, n % 32], v[r])
        check_decode(c, qr, after, out=o, lse=l)
    assert c.device_error() == 0


def test_two_threads():
    # two threads, a stream each, on one cache: appends to their own layers, then attention
    import threading
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    c, g = make(3, 8, 2, 64, 16, "bf16", "bf16", [500, 20, 0], layers=2, rotary=Rotary(64), extra_pages=1)
    c.pages[1] = c.pages[0]
    ins = [[tuple(torch.randn(3, h, 64, generator=g, device="cuda").bfloat16() for h in (8, 2, 2)) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(layer):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for q, k, v in ins[layer]:
                    qr = c.append(layer, k, v, q=q)
                    got[layer].append((qr, *c.decode(layer, qr, return_lse=True)))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 (told by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(layer,)) for layer in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for layer in range(2):
        for (q, k, v), (qr, out, lse) in zip(ins[layer], got[layer]):
            again = c.append(layer, k, v, q=q)
            assert torch.equal(again, qr)
            o2, l2 = c.decode(layer, again, return_lse=True)
            assert torch.equal(o2, out) and torch.equal(l2, lse)
        check_decode(c, qr, [501, 21, 1], layer=layer, out=out, lse=lse)


def test_streams():
    # a given stream, as an object and as a handle: results, and memory that is not handed out again early
    torch = T()
    c, q, k, v, after = small_step(3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
        qr = c.append(0, k, v, q=q, stream=stream)
        got = c.decode(0, qr, return_lse=True, stream=stream)
        rot = c.rotary.apply(c.lengths, q, stream=stream)
        junk = [torch.full_like(qr, 3.0) for _ in range(20)]      # on the current stream, meanwhile
        torch.cuda.synchronize()
        check_decode(c, qr, after, out=got[0], lse=got[1])
        assert torch.equal(rot, qr) and len(junk) == 20


def test_cache_refuses_what_the_binding_sees():
    torch = T()
    from tiered_kv_cache_int8_gb300 import HsError, PagedKVCache, Rotary
    c, q, k, v, _ = small_step()
    bad = [dict(k=k.half()), dict(k=k[:, :1]), dict(k=k[..., :64]), dict(v=v[:3]), dict(k=k.cpu()), dict(q=q[:3]), dict(q=q[:, :4]),
           dict(q=q, q_out=q[:2]), dict(tok_offsets=torch.zeros(3, device="cuda")), dict(q_out=q),
           dict(req_ids=torch.zeros(4, dtype=torch.int64, device="cuda"))]
    for kw in bad:
        a = dict(k=k, v=v)
        a.update(kw)
        with pytest.raises(ValueError):
            c.append(0, a.pop("k"), a.pop("v"), **a)
    with pytest.raises(HsError):
        c.append(1, k, v)
    with pytest.raises(HsError):      # 4 rows for 3 requests
        c.append(0, k, v, req_ids=torch.zeros(3, dtype=torch.int32, device="cuda"))
    for kw in (dict(q=q[:, :4]), dict(q=q.float()), dict(q=q, lengths=c.lengths.long()), dict(q=q, lengths=c.lengths[:2]),
               dict(q=q, out=q[:2]), dict(q=q, req_ids=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            c.decode(0, **kw)
    with pytest.raises(HsError):
        c.decode(-1, q)
    with pytest.raises(HsError):      # more requests than the cache has
        c.decode(0, torch.zeros(5, 8, 128, dtype=torch.bfloat16, device="cuda"))
    base = dict(n_layers=1, n_pages=4, page_size=16, max_requests=2, max_pages=2, h_q=4, h_kv=2, d=64)
    for kw in (dict(pages=torch.zeros(1, device="cuda")), dict(kv_scale=torch.zeros(1, device="cuda")),
               dict(dtype=torch.int32), dict(dtype=torch.float64)):
        with pytest.raises(ValueError):
            PagedKVCache(**{**base, **kw})
    for kw in (dict(d=96), dict(page_size=8), dict(h_q=5), dict(kv_dtype=torch.float16), dict(dtype=torch.float32), dict(n_pages=-1),
               dict(kv_dtype=torch.float8_e4m3fn)):
        with pytest.raises(HsError):
            PagedKVCache(**{**base, **kw})
    with pytest.raises(ValueError):
        PagedKVCache(**{**base, "max_requests": 4097, "pages": torch.zeros(2, device="cuda")})
    with pytest.raises(HsError):
        PagedKVCache(**base, rotary=Rotary(128)).append(0, k[:1, :, :64].contiguous(), v[:1, :, :64].contiguous())


def test_a_first_call_may_be_captured():
    # a process whose first calls of every kernel are inside a capture
    import subprocess
    import sys
    from tests.conftest import ROOT
    code = """
import torch
from tiered_kv_cache_int8_gb300 import PagedKVCache, Rotary
rot = Rotary(64)
c = PagedKVCache(n_layers=1, n_pages=8, page_size=16, max_requests=2, max_pages=4, h_q=4, h_kv=2, d=64, rotary=rot)
c.reserve(0, 20); c.reserve(1, 1)
k = torch.randn(2, 2, 64, device="cuda").bfloat16(); q = torch.randn(2, 4, 64, device="cuda").bfloat16()
pos = torch.zeros(2, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    x = rot.apply(pos, q)
    qr = c.append(0, k, k, q=q)
    o = c.decode(0, qr)
g.replay(); torch.cuda.synchronize()
assert torch.equal(x, q) and torch.equal(qr, q) and c.device_error() == 0
assert torch.equal(o, k.repeat_interleave(2, dim=1))
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_decode_of_the_most_requests():
    torch = T()
    R, d, page = 4096, 64, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    c = PagedKVCache(n_layers=1, n_pages=R, page_size=page, max_requests=R, max_pages=1, h_q=3, h_kv=1, d=d)
    c.pages.copy_(filled(c.pages.shape, torch.bfloat16, g, False))
    c.page_table[:, 0] = torch.randperm(R, generator=g, device="cuda").to(torch.int32)
    lengths = torch.randint(0, page + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
    c.set_lengths(lengths)
    q = torch.randn(R, 3, d, generator=g, device="cuda").bfloat16()
    out, lse = c.decode(0, q, return_lse=True)
    kv = c.pages[0][c.page_table[:, 0].long(), :, 0].double()               # [R, 2, page, d]
    seen = torch.arange(page, device="cuda")[None] < lengths[:, None]
    s = torch.einsum("rhd,rnd->rhn", q.double(), kv[:, 0]) / math.sqrt(d)
    s = torch.where(seen[:, None], s, -math.inf)
    p = torch.nan_to_num(torch.softmax(s, -1))
    want = torch.einsum("rhn,rnd->rhd", p, kv[:, 1])
    size = torch.einsum("rhn,rnd->rhd", p, kv[:, 1].abs())
    # scores of 64 products each, at most 16 of them; weights and output rounded as in paged_plain.attend
    dots = torch.einsum("rhd,rnd->rhn", q.double().abs(), kv[:, 0].abs()).amax(-1, keepdim=True) / math.sqrt(d)
    tol = size * (2.0 ** -8 + 2 * (d + 8) * 2.0 ** -23 * dots + 2.0 ** -16) + 2.0 ** -20 * want.abs()
    within(out, want, tol + 2.0 ** -8 * (want.abs() + tol) + plain.TINY[q.dtype], "out")
    some = lengths > 0
    within(lse[some], torch.logsumexp(s[some], -1), ((d + 8) * 2.0 ** -23 * dots[some, :, 0] + 2.0 ** -16), "lse")
    assert (lse[~some] == -math.inf).all() and (~some).any() and c.device_error() == 0


def test_decode_in_place_and_repeated_ids():
    torch = T()
    from tiered_kv_cache_int8_gb300 import HsError
    lengths = [3000, 17, 0, 400]
    c, g = make(4, 40, 2, 128, 32, "bf16", "bf16", lengths)
    q = torch.randn(6, 40, 128, generator=g, device="cuda").bfloat16()
    ids = [0, 3, 0, 1, 2, 0]
    i32 = torch.tensor(ids[:4], dtype=torch.int32, device="cuda")
    out, lse = check_decode(c, q[:4].contiguous(), lengths, ids=ids[:4])
    x = q[:4].clone()
    assert c.decode(0, x, req_ids=i32, out=x) is x and torch.equal(x, out)
    with pytest.raises(HsError):
        c.decode(0, q[:4], req_ids=i32, out=q[1:5])
    # a single request's query with any stride
    wide = torch.randn(1, 41 * 128 + 3, generator=g, device="cuda").bfloat16()
    check_decode(c, wide[:, :40 * 128].view(1, 40, 128), lengths, ids=[3])


@pytest.mark.parametrize("offsets", [False, True])
def test_append_of_no_tokens(offsets):
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    c, g = make(3, 2, 1, 64, 16, "bf16", "e4m3", [3, 0, 20], rotary=Rotary(64))
    c.next_lengths.fill_(-7)
    before = c.pages.view(torch.uint8).clone()
    none = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    nq = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    kw = dict(tok_offsets=torch.zeros(4, dtype=torch.int32, device="cuda")) if offsets else dict(
        req_ids=torch.arange(3, dtype=torch.int32, device="cuda"))
    assert c.append(0, none, none, q=nq, **kw).shape == (0, 2, 64)
    assert c.next_lengths.tolist() == [3, 0, 20] and torch.equal(c.pages.view(torch.uint8), before)
    assert c.device_error() == 0


def test_the_two_tier_cache_takes_rotated_rows():
    # the rotation feeds the two-tier cache: rows and queries rotated by it give the attention of rotated rows
    torch = T()
    from oracle import sparse_attention
    from tests.harness import MAX_ABS, REL_L2, attention_error
    from tiered_kv_cache_int8_gb300 import HiSparseCache, Rotary
    g = torch.Generator(device="cuda").manual_seed(9)
    n, hq, hk, d = 60, 8, 2, 128
    c = HiSparseCache(n_layers=1, max_requests=1, max_context=64, h_q=hq, h_kv=hk, d_qk=d, d_v=d, d_idx=64, top_k=64, hot_slots=64)
    R = Rotary(d)
    rows = torch.randn(1, n, 2 * hk * d, generator=g, device="cuda").bfloat16()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    k = rows[0, :, :hk * d].view(n, hk, d)
    R.apply(pos, k, out=k)
    c.append(0, rows, torch.randint(-127, 128, (1, n, 64), generator=g, device="cuda", dtype=torch.int8))
    q = torch.randn(1, hq, d, generator=g, device="cuda").bfloat16()
    qr = R.apply(pos[-1:], q)
    out = c.decode_layer(0, torch.zeros(1, 64, dtype=torch.int8, device="cuda"), qr)
    as_bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)   # noqa: E731
    ref = sparse_attention(as_bits(qr[0]), as_bits(rows[0]), h_kv=hk, d_qk=d, d_v=d, v_offset=hk * d)
    ma, rel = attention_error(as_bits(out[0]), ref)
    assert ma <= MAX_ABS and rel <= REL_L2
    c.close()


def test_append_over_more_threads_than_31_bits_count():
    # one-element accesses of broadcast rows, most of which belong to nobody: 9 million CTAs of 256 threads
    torch = T()
    from tiered_kv_cache_int8_gb300 import PagedKVCache, Rotary
    n, hk, d, page = 140000, 1024, 64, 16
    assert n * 2 * (hk // 4) // 8 * 256 > 1 << 31
    c = PagedKVCache(n_layers=1, n_pages=3, page_size=page, max_requests=2, max_pages=2, h_q=hk, h_kv=hk, d=d, rotary=Rotary(2))
    c.pages.zero_()
    c.page_table.copy_(torch.tensor([[2, 0], [1, -1]], dtype=torch.int32))
    c.set_lengths(torch.tensor([15, 3], dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(11)
    k, v = (torch.randn(1, 1, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    c.append(0, k.expand(n, hk, d), v.expand(n, hk, d), tok_offsets=torch.tensor([5, 7, 8], dtype=torch.int32, device="cuda"))
    assert c.next_lengths.tolist() == [17, 4] and c.lengths.tolist() == [15, 3] and c.device_error() == 0
    at = {(2, 15): 15, (0, 0): 16, (1, 3): 3}           # (page, slot): position
    for (p, slot), pos in at.items():
        want, tol = plain.rotate(k, torch.tensor([pos], device="cuda"), plain.frequencies(2))
        got = c.pages[0, p, :, :, slot].clone()
        within(got[0], want[0].expand(hk, d), (tol + 2.0 ** -8 * (want.abs() + tol) + plain.TINY[k.dtype])[0].expand(hk, d), "keys")
        assert torch.equal(got[1], v[0].expand(hk, d))
        c.pages[0, p, :, :, slot] = 0
    assert not c.pages.any()


def test_outputs_over_another_tensor_are_refused():
    torch = T()
    from tiered_kv_cache_int8_gb300 import HsError, Rotary
    n, h, d = 9, 4, 64
    R = Rotary(d)
    g = torch.Generator(device="cuda").manual_seed(12)
    pos = torch.arange(3, 3 + n, dtype=torch.int32, device="cuda")
    qkv = torch.randn(n, h, 3, d, generator=g, device="cuda").bfloat16()    # queries, keys and values of a head together
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    want = R.apply(pos, q, k)
    before = qkv.clone()
    for out in ((k, q), (q, q), (torch.empty_like(want[0]),) * 2, (q, q[:, :, :]), (k, torch.empty_like(want[0]))):
        with pytest.raises(HsError):
            R.apply(pos, q, k, out=out)
    with pytest.raises(HsError):
        R.apply(pos, q, q, out=(q, torch.empty_like(want[0])))
    assert torch.equal(qkv, before)
    R.apply(pos, q, k, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 2], before[:, :, 2])
    c, cq, ck, cv, _ = small_step(2)
    out = ck.repeat(1, 4, 1)
    with pytest.raises(HsError):
        c.append(0, out[:, :2], cv, q=cq, q_out=out)
    with pytest.raises(HsError):
        c.append(0, ck, out[:, 6:], q=cq, q_out=out)
    assert c.device_error() == 0 and not c.next_lengths.ne(c.lengths).any()


def test_gradients_are_not_dropped_silently():
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    n, h, d = 6, 2, 64
    R = Rotary(d)
    g = torch.Generator(device="cuda").manual_seed(13)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    x, y = (torch.randn(n, h, d, generator=g, device="cuda") for _ in range(2))
    leaf = x.clone().requires_grad_()
    want = R.apply(pos, x, y)
    for args, kw in (((leaf,), {}), ((x, leaf), {}), ((leaf, x), {}), ((x,), dict(out=leaf)), ((x, y), dict(out=(torch.empty_like(x), leaf))),
                     ((leaf * 2,), {}), ((leaf,), dict(stream=torch.cuda.current_stream()))):
        with pytest.raises(ValueError):
            R.apply(pos, *args, **kw)
    assert torch.equal(leaf.detach(), x)
    with torch.no_grad():
        assert torch.equal(R.apply(pos, leaf, y)[0], want[0])
    with torch.inference_mode():
        z = x.clone()
        assert torch.equal(R.apply(pos, z, out=z), want[0])
    assert torch.equal(R.apply(pos, leaf.detach()), want[0])

    class Rotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            return R.apply(pos, t)

        @staticmethod
        def backward(ctx, up):
            return R.apply(pos, up, transpose=True)

    Rotate.apply(leaf).backward(y)
    assert torch.equal(leaf.grad, R.apply(pos, y, transpose=True))
    # a tensor that a backward pass still needs, written in place
    weight = torch.ones_like(x, requires_grad=True)
    for write in (lambda t: R.apply(pos, t, out=t), lambda t: R.apply(pos, t, x, out=(t, torch.empty_like(x))),
                  lambda t: R.apply(pos, x, t, out=(torch.empty_like(x), t))):
        t = y.clone()
        loss = (t * weight).sum()
        write(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    c, q, k, v, _ = small_step(5)
    weight = torch.ones_like(q, requires_grad=True)
    for write in (lambda t: c.append(0, k, v, q=t, q_out=t), lambda t: c.decode(0, q, out=t)):
        t = q.clone()
        loss = (t * weight).sum()
        write(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_refusals_on_a_given_stream():
    # the same errors as on the current stream
    torch = T()
    c, q, k, v, _ = small_step(6)
    s = torch.cuda.Stream()
    for call in (lambda: c.rotary.apply(c.lengths.cpu(), q, stream=s), lambda: c.rotary.apply(c.lengths, q.cpu(), stream=s),
                 lambda: c.append(0, k.cpu(), v, stream=s), lambda: c.decode(0, q.cpu(), stream=s),
                 lambda: c.decode(0, q, lengths=c.lengths.cpu(), stream=s.cuda_stream)):
        with pytest.raises(ValueError):
            call()
    assert torch.cuda.current_stream() != s and c.device_error() == 0


# ---- wide tables: the work is shared out evenly and its pieces joined, however short the contexts are ----------

def widened(c, positions=1040):
    """The same requests over the same pool with a table of at least `positions` positions (its further columns hold -1)."""
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    w = PagedKVCache(n_layers=c.n_layers, n_pages=c.n_pages, page_size=c.page_size, max_requests=c.max_requests,
                     max_pages=max(c.max_pages, -(-positions // c.page_size)), h_q=c.h_q, h_kv=c.h_kv, d=c.d, dtype=c.dtype,
                     kv_dtype=c.kv_dtype, softmax_scale=c.cfg.softmax_scale, window=c.cfg.window, rotary=c.rotary,
                     kv_scale=c.kv_scale, pages=c.pages)
    w.page_table[:, :c.max_pages].copy_(c.page_table)
    w.set_lengths(c.lengths)
    return w


RAGGED = [(37 * r) % 90 for r in range(150)]
RAGGED[3], RAGGED[77], RAGGED[149] = 4000, 1500, 1041


@pytest.mark.parametrize("lengths", [[1] * 300, list(range(200)), RAGGED, [0] * 128 + [5], [17] * 129, [0, 1, 15, 16, 17, 65, 130]],
                         ids=["ones", "rising", "ragged", "mostly empty", "alike", "few"])
@pytest.mark.parametrize("typ, kv, hq, hk, d", [("bf16", "bf16", 6, 2, 64), ("fp16", "e4m3", 8, 1, 128), ("bf16", "bf16", 20, 1, 256),
                                                ("fp16", "fp16", 3, 3, 64)])
def test_wide_tables_of_short_contexts(lengths, typ, kv, hq, hk, d):
    torch = T()
    c, g = make(len(lengths), hq, hk, d, 16, typ, kv, lengths, seed=len(lengths) + d)
    c = widened(c)
    q = torch.randn(len(lengths), hq, d, generator=g, device="cuda").to(dtype(typ))
    out, lse = check_decode(c, q, lengths)
    again, lse2 = c.decode(0, q, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2) and c.device_error() == 0


@pytest.mark.parametrize("typ, kv", [("bf16", "bf16"), ("fp16", "e4m3")])
@pytest.mark.parametrize("window", [1009, 1024, 2000])
def test_wide_tables_with_a_window(typ, kv, window):
    torch = T()
    lengths = [0, 1, 17, window - 1, window, window + 1, 5000, 0, 2500, 40]
    c, g = make(len(lengths), 8, 4, 64, 32, typ, kv, lengths, window=window)
    q = torch.randn(len(lengths), 8, 64, generator=g, device="cuda").to(dtype(typ))
    raw = c.pages.view(torch.uint8) if kv == "e4m3" else c.pages
    for r, n in enumerate(lengths):
        pos = torch.arange(max(0, n - window), device="cuda")       # not used, whatever they hold
        raw[0][c.page_table[r][pos // 32].long(), :, :, pos % 32] = 0x7F if kv == "e4m3" else math.nan
    check_decode(c, q, lengths, window=window)
    assert c.device_error() == 0


def test_wide_tables_skip_bad_requests():
    torch = T()
    from tiered_kv_cache_int8_gb300 import hs
    R = 140                                    # more than a warp looks through by itself
    lengths = [(53 * r) % 200 for r in range(R)]
    lengths[7] = 1300
    c, g = make(R, 4, 2, 64, 16, "bf16", "bf16", lengths, max_requests=R + 1)
    c = widened(c)
    for n in (20, R):                          # few requests, many
        q = torch.randn(n, 4, 64, generator=g, device="cuda").bfloat16()
        ids = list(range(n))
        ids[1], ids[n - 2], ids[9] = R + 1, -1, 7
        c._error.zero_()
        out, lse = c.decode(0, q, req_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"), return_lse=True)
        assert c.device_error() == hs.HS_DEVERR_REQ_RANGE
        bad = [1, n - 2]
        fine = [i for i in range(n) if i not in bad]
        assert (out[bad] == 0).all() and (lse[bad] == -math.inf).all()
        check_decode(c, q[fine].contiguous(), lengths, ids=[ids[i] for i in fine], out=out[fine], lse=lse[fine])
        # lengths outside the table
        other = list(lengths) + [0]
        other[0], other[5] = -3, c.max_pages * 16 + 1
        c._error.zero_()
        out, lse = c.decode(0, q, lengths=torch.tensor(other, dtype=torch.int32, device="cuda"), return_lse=True)
        assert c.device_error() == hs.HS_DEVERR_CAPACITY
        assert (out[[0, 5]] == 0).all() and (lse[[0, 5]] == -math.inf).all()
        fine = [i for i in range(n) if i not in (0, 5)]
        check_decode(c, q[fine].contiguous(), lengths, ids=fine, out=out[fine], lse=lse[fine])


@pytest.mark.parametrize("typ, kv, hq, hk", [("bf16", "bf16", 4, 1), ("fp16", "e4m3", 8, 2)])
def test_bad_pages_over_whole_shares(typ, kv, hq, hk):
    # pieces in which nothing is attended, alone and joined with others
    torch = T()
    from tiered_kv_cache_int8_gb300 import hs
    lengths = [60000, 30000, 5000, 64]
    c, g = make(4, hq, hk, 64, 64, typ, kv, lengths)
    q = torch.randn(4, hq, 64, generator=g, device="cuda").to(dtype(typ))
    for bad in ([(0, 200, 600)], [(0, 0, 700), (1, 100, 469)], [(0, 1, 938), (1, 0, 469), (2, 0, 79)], [(r, 0, 938) for r in range(4)]):
        held = c.page_table.clone()
        for r, a, b in bad:
            c.page_table[r, a:b] = c.n_pages + 5 if r % 2 else -1
        c._error.zero_()
        out, lse = c.decode(0, q, return_lse=True)
        assert c.device_error() == hs.HS_DEVERR_PAGE
        for r in range(4):
            want, wl, tol, tl = plain.attend(q[r], c.pages[0], c.page_table[r], lengths[r], 0, 1 / 8,
                                             None if c.kv_scale is None else c.kv_scale[0])
            within(out[r], want, tol, f"out of request {r}")
            if torch.isinf(wl).all():
                assert (lse[r] == -math.inf).all() and (out[r] == 0).all()
            else:
                within(lse[r], wl, tl, f"lse of request {r}")
        c.page_table.copy_(held)


def test_only_empty_requests_over_a_used_workspace():
    # the pieces and chains that an earlier call left behind are not taken up
    import ctypes
    torch = T()
    from tiered_kv_cache_int8_gb300 import hs
    c, g = make(2, 8, 2, 64, 64, "bf16", "bf16", [40000, 3])
    q = torch.randn(2, 8, 64, generator=g, device="cuda").bfloat16()
    ws = torch.full((c._ws_bytes,), 0x7F, dtype=torch.uint8, device="cuda")
    heads = hs.HsHeads(q.data_ptr(), 8 * 64, 64, 8, 0)

    def run(lengths):
        lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(q, 7.0), torch.full((2, 8), 7.0, device="cuda")
        rc = hs.lib().hs_paged_decode(c._h, 0, 2, None, c.page_table.data_ptr(), lens.data_ptr(), ctypes.byref(heads), out.data_ptr(),
                                      lse.data_ptr(), ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        return out, lse

    for lengths in ([40000, 3], [0, 0], [40000, 3], [3, 0], [0, 3], [39999, 0]):
        out, lse = run(lengths)
        check_decode(c, q, lengths, out=out, lse=lse)
    assert c.device_error() == 0


@pytest.mark.parametrize("typ, kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("wide", [False, True])
def test_a_row_that_wins_alone(typ, kv, wide):
    # large scores that are exact in 32 bits (integers below 2^24 under a power of two); the second best is 200 or more
    # below, so its weight is 0 and the output is the winner's row
    torch = T()
    lengths = [1, 2, 17, 100, 500, 1000, 900]
    at = [0, 1, 16, 0, 499, 480, 16]                     # the winners' positions
    c, g = make(len(lengths), 4, 2, 64, 64, typ, kv, lengths, scale=0.125)
    if kv == "e4m3":
        c.kv_scale.copy_(2.0 ** torch.randint(-6, 3, c.kv_scale.shape, generator=g, device="cuda").float())
    if wide:
        c = widened(c)
    big = 4096.0
    q = (torch.randint(0, 2, (len(lengths), 4, 64), generator=g, device="cuda") * 2 - 1) * big
    q[:, 1::2] = q[:, ::2]                               # the heads of a group look for the same row
    raw = c.pages.view(torch.uint8) if kv == "e4m3" else c.pages
    bits = (lambda x: x.to(c.kv_dtype).view(torch.uint8)) if kv == "e4m3" else (lambda x: x.to(c.kv_dtype))
    for r, n in enumerate(lengths):
        pos = torch.arange(n, device="cuda")
        for h in range(2):
            sign = q[r, 2 * h] / big
            rows = torch.randint(-1, 2, (n, 64), generator=g, device="cuda").float()
            rows = rows * torch.where(rows * sign > 0, 0.0, 1.0)              # products of 0 or below
            rows[at[r]] = 3 * sign                                            # 3 * 4096 * 64
            raw[0][c.page_table[r][pos // 64].long(), 0, h, pos % 64] = bits(rows)
    out, lse = c.decode(0, q.to(dtype(typ)), return_lse=True)
    for r, n in enumerate(lengths):
        kv_row = c.pages[0, c.page_table[r, at[r] // 64].long(), :, :, at[r] % 64].double()      # [2, hk, d]
        scales = torch.ones(2, 2, dtype=torch.float64, device="cuda") if kv != "e4m3" else c.kv_scale[0].double()
        v = (kv_row[1] * scales[1][:, None]).repeat_interleave(2, dim=0)
        if kv == "e4m3":
            # the winner's weight is rounded to fp16, its share of the sum is not; then products and the output
            tol = v.abs() * (2.0 ** -11 + 2.0 ** -20)
            within(out[r], v, tol + plain.HALF_STEP[dtype(typ)] * (v.abs() + tol) + plain.TINY[dtype(typ)], f"out of request {r}")
        else:
            # a weight in two parts is off by 2^-16 at most: the row itself is the nearest value
            assert torch.equal(out[r].double(), v), f"out of request {r}"
        s = (3 * big * 64 * 0.125 * scales[0])[:, None].expand(2, 2).reshape(4)
        within(lse[r], s, s * 2.0 ** -21, f"lse of request {r}")
    assert c.device_error() == 0


@pytest.mark.parametrize("width", [1, 66])
def test_the_most_requests_with_weights_in_two_parts(width):
    torch = T()
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    R, d, page = 4096, 64, 16
    g = torch.Generator(device="cuda").manual_seed(21)
    c = PagedKVCache(n_layers=1, n_pages=R, page_size=page, max_requests=R, max_pages=width, h_q=3, h_kv=1, d=d)
    c.pages.copy_(filled(c.pages.shape, torch.bfloat16, g, False))
    c.page_table[:, 0] = torch.randperm(R, generator=g, device="cuda").to(torch.int32)
    lengths = torch.randint(0, page + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
    c.set_lengths(lengths)
    q = torch.randn(R, 3, d, generator=g, device="cuda").bfloat16()
    out, lse = c.decode(0, q, return_lse=True)
    kv = c.pages[0][c.page_table[:, 0].long(), :, 0].double()               # [R, 2, page, d]
    seen = torch.arange(page, device="cuda")[None] < lengths[:, None]
    s = torch.einsum("rhd,rnd->rhn", q.double(), kv[:, 0]) / math.sqrt(d)
    s = torch.where(seen[:, None], s, -math.inf)
    p = torch.nan_to_num(torch.softmax(s, -1))
    want = torch.einsum("rhn,rnd->rhd", p, kv[:, 1])
    size = torch.einsum("rhn,rnd->rhd", p, kv[:, 1].abs())
    # as paged_plain.attend has it, for at most 16 positions: a weight in two parts of 2^-8 each
    dots = torch.einsum("rhd,rnd->rhn", q.double().abs(), kv[:, 0].abs()).amax(-1, keepdim=True) / math.sqrt(d)
    e_s = (d + 8) * 2.0 ** -23 * dots + 2.0 ** -22 * dots
    e_p = 2 * e_s + 2.0 ** -20 + (page + 64) * 2.0 ** -23
    tol = size * (plain.HALF_STEP[q.dtype] ** 2 + e_p) + 2.0 ** -20 * want.abs()
    within(out, want, tol + plain.HALF_STEP[q.dtype] * (want.abs() + tol) + plain.TINY[q.dtype], "out")
    some = lengths > 0
    within(lse[some], torch.logsumexp(s[some], -1), (e_s + 2.0 ** -20 + (page + 64) * 2.0 ** -24)[some, :, 0] + 2.0 ** -20, "lse")
    assert (lse[~some] == -math.inf).all() and (out[~some] == 0).all() and c.device_error() == 0


def test_rotary_takes_an_output_for_each_input():
    torch = T()
    from tiered_kv_cache_int8_gb300 import Rotary
    R = Rotary(64)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    x, y = (torch.randn(4, 2, 64, device="cuda") for _ in range(2))
    a, b, c = (torch.full_like(x, 7.0) for _ in range(3))
    for args, out in (((x, y), (a, b, c)), ((x, y), (a,)), ((x, y), a), ((x,), (a, b)), ((x,), ()), ((x, y), ())):
        with pytest.raises(ValueError):
            R.apply(pos, *args, out=out)
    assert (a == 7.0).all() and (b == 7.0).all()
    assert R.apply(pos, x, out=(a,)) is a and torch.equal(a, R.apply(pos, x))
    got = R.apply(pos, x, y, out=[b, c])
    assert got[0] is b and got[1] is c and torch.equal(c, R.apply(pos, y))
