"""Prompt attention over the paged cache, scores with a cap or a distance bias, 4-bit pages
and rows read back, on the GPU, against plain 64-bit implementations (tests/paged_more.py,
which also derives the tolerances).  Rows that a call must not use hold NaN."""
import math

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


def M():
    from tests import paged_more
    return paged_more


def ints(x):
    torch = T()
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(new, first=0):
    out = [first]
    for n in new:
        out.append(out[-1] + n)
    return ints(out)


def queries(n, hq, d, typ, seed=0):
    # some heads look closely, some broadly
    torch = T()
    g = torch.Generator(device="cuda").manual_seed(seed + 101)
    sharp = torch.rand(1, hq, 1, generator=g, device="cuda") * 3 + 0.5
    return (torch.randn(n, hq, d, generator=g, device="cuda") * sharp).to(M().DT[typ])


def check_attend(c, q, held, new, *, layer=0, prefix=None, scale=None, ids=None, got=None):
    torch, pm = T(), M()
    ids = list(range(len(new))) if ids is None else ids
    if got is None:
        got = c.attend(layer, q, tok_offsets=offsets(new), prefix=None if prefix is None else ints(prefix), return_lse=True,
                       req_ids=ints(ids))
    out, lse = got
    at = 0
    for i, r in enumerate(ids):
        rows = slice(at, at + new[i])
        at += new[i]
        pos = torch.arange(held[r], held[r] + new[i], device="cuda")
        want, wl, tol, tl = pm.attend(c, layer, r, q[rows], pos, held[r] + new[i], prefix=0 if prefix is None else prefix[r], scale=scale)
        pm.within(lse[rows], wl, tl, f"lse of request {r}")
        pm.within(out[rows], want, tol, f"out of request {r}")
    return out, lse


def attended(R, hq, hk, d, page, typ, kv, held, new, *, seed=0, bias=False, prefix=None, **kw):
    pm = M()
    c = pm.make(R, hq, hk, d, page, typ, kv, [a + b for a, b in zip(held, new)], seed=seed, slopes=pm.slopes_of(hq) if bias else None,
                **kw)
    c.set_lengths(ints(held))
    q = queries(sum(new), hq, d, typ, seed)
    got = check_attend(c, q, held, new, prefix=prefix)
    assert c.device_error() == 0
    return c, q, got


KINDS = [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3"), ("bf16", "int4"), ("fp16", "int4")]


# ---- prompt attention -----------------------------------------------------------------------------

@pytest.mark.parametrize("typ, kv", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq, hk, page", [(4, 4, 16), (8, 1, 64), (12, 4, 32), (32, 2, 128), (40, 1, 256), (7, 1, 16)])
def test_attend_lengths_and_heads(typ, kv, d, hq, hk, page):
    held, new = [0, 0, 17, 0, 300, 64, 127, 5], [1, 129, 16, 0, 3, 64, 1, 200]
    attended(len(held), hq, hk, d, page, typ, kv, held, new, seed=d + hq)


@pytest.mark.parametrize("typ, kv, d, hq, hk", [("bf16", "bf16", 128, 8, 2), ("fp16", "e4m3", 64, 6, 2), ("bf16", "int4", 256, 4, 1),
                                                ("fp16", "fp16", 256, 3, 3), ("bf16", "int4", 128, 8, 2)])
@pytest.mark.parametrize("window, softcap, bias, prefix", [
    (1, 0.0, False, None), (16, 0.0, False, None), (100, 30.0, False, None), (257, 0.0, True, None), (5000, 0.0, False, None),
    (0, 2.0, True, [0, 250, 1000, 7]), (0, 0.0, False, [1, 129, 64, 0]), (60, 50.0, True, [200, 10, 0, 400]), (0, 0.0, True, None),
])
def test_attend_masks_and_scores(typ, kv, d, hq, hk, window, softcap, bias, prefix):
    attended(4, hq, hk, d, 32, typ, kv, [0, 100, 333, 0], [260, 150, 17, 128], window=window, softcap=softcap, bias=bias, prefix=prefix,
             seed=window)


@pytest.mark.parametrize("typ, kv, d, hq, hk", [("bf16", "bf16", 128, 8, 1), ("bf16", "bf16", 64, 4, 2), ("fp16", "int4", 256, 4, 2),
                                                ("bf16", "e4m3", 128, 16, 2)])
@pytest.mark.parametrize("held, new", [([20000], [5]), ([9000, 3], [1, 2]), ([0], [1]), ([4000] * 3, [40] * 3), ([1000], [700])])
def test_attend_splits(typ, kv, d, hq, hk, held, new):
    # few rows over long contexts: work shared by all CTAs and joined
    attended(len(held), hq, hk, d, 64, typ, kv, held, new, seed=sum(new))


@pytest.mark.parametrize("typ, kv, d", [("bf16", "bf16", 128), ("fp16", "fp16", 64), ("bf16", "int4", 128)])
def test_attend_many_requests(typ, kv, d):
    # more segments than CTAs, most of one token, some without any
    new = [(i * 7) % 4 for i in range(700)]
    held = [(i * 13) % 90 for i in range(700)]
    attended(700, 4, 2, d, 16, typ, kv, held, new)


def test_attend_the_most_requests():
    attended(4096, 2, 1, 64, 16, "bf16", "bf16", [i % 40 for i in range(4096)], [1 + (i % 5 == 0) for i in range(4096)])


def test_attend_long_prompt_of_whole_and_cut_segments():
    attended(2, 4, 1, 128, 128, "bf16", "bf16", [0, 900], [2500, 1111], seed=3)


def test_attend_one_token_is_decode():
    # the same positions attended by both calls, cap and bias too
    torch, pm = T(), M()
    held = [0, 31, 700, 1999]
    for kv in ("bf16", "int4"):
        c = pm.make(4, 8, 2, 128, 32, "bf16", kv, [n + 1 for n in held], softcap=20.0, slopes=pm.slopes_of(8))
        q = queries(4, 8, 128, "bf16")
        c.set_lengths(ints(held))
        a, la = c.attend(0, q, return_lse=True)
        c.set_lengths(ints([n + 1 for n in held]))
        b, lb = c.decode(0, q, return_lse=True)
        for r in range(4):
            want, wl, tol, tl = pm.attend(c, 0, r, q[r:r + 1], ints([held[r]]).long(), held[r] + 1)
            _, _, tight, _ = pm.attend(c, 0, r, q[r:r + 1], ints([held[r]]).long(), held[r] + 1, one=True)
            pm.within(a[r:r + 1], want, tol, "attend")
            pm.within(b[r:r + 1], want, tight, "decode")
            pm.within(la[r:r + 1], wl, tl, "lse")
            pm.within(lb[r:r + 1], wl, tl, "lse")


def test_attend_skips_bad_requests_pages_and_offsets():
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import hs
    for kv in ("bf16", "int4", "e4m3"):
        c = pm.make(6, 4, 2, 128, 32, "bf16", kv, [200, 100, 90, 64, 40, 300], extra_pages=1)
        held = [150, 90, 0, 60, 30, 100]
        new = [50, 10, 90, 4, 10, 200]
        c.set_lengths(ints(held))
        q = queries(sum(new) + 5, 4, 128, "bf16")
        # a bad id, a negative length, a page out of range, rows of nobody in front and behind
        ids = ints([0, 77, 2, 3, 4, 5])
        c.lengths[3] = -2
        c.page_table[5, 1] = c.n_pages
        c.page_table[5, 4] = -9
        offs = offsets(new, 2)
        out = torch.full((sum(new) + 5, 4, 128), 7.0, device="cuda").bfloat16()
        got, lse = c.attend(0, q, req_ids=ids, tok_offsets=offs, out=out, return_lse=True)
        assert got is out
        assert c.device_error() == hs.HS_DEVERR_REQ_RANGE | hs.HS_DEVERR_CAPACITY | hs.HS_DEVERR_PAGE
        at = offs.tolist()
        assert (out[:2] == 7).all() and (out[at[-1]:] == 7).all()
        for i in (1, 3):
            assert (out[at[i]:at[i + 1]] == 0).all() and (lse[at[i]:at[i + 1]] == -math.inf).all()
        for i in (0, 2, 4, 5):
            rows = slice(at[i], at[i + 1])
            pos = torch.arange(held[i], held[i] + new[i], device="cuda")
            want, wl, tol, tl = pm.attend(c, 0, i, q[rows], pos, held[i] + new[i])
            pm.within(lse[rows], wl, tl, f"lse {i}")
            pm.within(out[rows], want, tol, f"out {i}")
        # offsets that fall, or leave the rows: no tokens for their request
        c._error.zero_()
        c.lengths[3] = 60
        out.fill_(7.0)
        c.attend(0, q, tok_offsets=ints([0, 50, 40, 40, 44, 54, 9999]), out=out)
        assert c.device_error() & hs.HS_DEVERR_OFFSETS
        assert (out[54:] == 7).all()


def test_attend_offsets_that_claim_rows_twice():
    # decreasing offsets may give many requests the same rows: refused as a whole (the work would have no bound)
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import hs
    for d, kv in ((64, "bf16"), (128, "int4"), (256, "bf16")):
        R, n = 9, 150
        c = pm.make(R, 4, 2, d, 32, "bf16", kv, [n] * R)
        c.set_lengths(ints([0] * R))
        q = queries(n, 4, d, "bf16")
        out = torch.full((n, 4, d), 7.0, device="cuda").bfloat16()
        twice = ints([0, n] * 5)
        ids = ints([0, 1, 2, 3, 77, 5, 6, 7, 8])                  # (a bad request's rows are not cleared either)
        c.attend(0, q, req_ids=ids, tok_offsets=twice, out=out)
        assert c.device_error() == hs.HS_DEVERR_OFFSETS | hs.HS_DEVERR_REQ_RANGE
        assert (out == 7).all()
        # where the rows suffice, requests with sound offsets keep theirs
        c._error.zero_()
        some = [0, 20, 999, 30, 60, 60, 140, 140, 140, 140]
        got, lse = c.attend(0, q, tok_offsets=ints(some), out=out, return_lse=True)
        assert c.device_error() == hs.HS_DEVERR_OFFSETS
        assert (out[20:30] == 7).all() and (out[140:] == 7).all()
        for r in (0, 3, 5):
            rows = slice(some[r], some[r + 1])
            check_attend(c, q[rows], [0] * R, [some[r + 1] - some[r]], ids=[r], got=(out[rows], lse[rows]))
        check_attend(c, q, [0] * R, [n], ids=[4])


def test_attend_where_nothing_is_seen():
    # every page of a request out of range: rows of zeros
    torch, pm = T(), M()
    for kv in ("fp16", "int4"):
        c = pm.make(2, 4, 1, 64, 16, "fp16", kv, [70, 50])
        c.set_lengths(ints([20, 10]))
        c.page_table[0] = -1
        q = queries(90, 4, 64, "fp16")
        out, lse = c.attend(0, q, tok_offsets=ints([0, 50, 90]), return_lse=True)
        assert (out[:50] == 0).all() and (lse[:50] == -math.inf).all()
        check_attend(c, q[50:], [20, 10], [40], ids=[1], got=(out[50:], lse[50:]))


def test_attend_released_pages_behind_the_window():
    # positions that the window has left behind may have no page any more
    torch, pm = T(), M()
    for kv in ("bf16", "e4m3"):
        c = pm.make(1, 4, 2, 128, 16, "bf16", kv, [600], window=100)
        c.set_lengths(ints([500]))
        q = queries(100, 4, 128, "bf16")
        want = c.attend(0, q, tok_offsets=ints([0, 100]), return_lse=True)
        c.page_table[0, :(500 - 99) // 16] = -1
        got = c.attend(0, q, tok_offsets=ints([0, 100]), return_lse=True)
        assert c.device_error() == 0
        check_attend(c, q, [500], [100], got=got)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attend_strides_scale_layers_and_in_place():
    torch, pm = T(), M()
    held, new, hq, hk, d = [40, 0], [30, 100], 6, 2, 128
    c = pm.make(2, hq, hk, d, 64, "bf16", "bf16", [70, 100], layers=3, layer=2, scale=0.3)
    c.set_lengths(ints(held))
    wide = torch.randn(130, (hq + 2 * hk) * d, device="cuda").bfloat16()
    q = wide[:, :hq * d].view(130, hq, d)
    out, lse = check_attend(c, q, held, new, layer=2, scale=0.3)
    by_heads = q.transpose(0, 1).contiguous().transpose(0, 1)
    again = c.attend(2, by_heads, tok_offsets=offsets(new))
    assert torch.equal(again, out)
    mine = q.contiguous()
    assert c.attend(2, mine, tok_offsets=offsets(new), out=mine) is mine
    assert torch.equal(mine, out)
    # one request's tokens without offsets
    one = pm.make(1, hq, hk, d, 64, "bf16", "bf16", [77])
    one.set_lengths(ints([7]))
    check_attend(one, q[:70], [7], [70], got=one.attend(0, q[:70], req_ids=ints([0]), return_lse=True))


def test_attend_values_at_the_border():
    # infinite and NaN keys and values behind the tokens' last position, in the same pages
    torch, pm = T(), M()
    for bad in (math.nan, math.inf, -math.inf):
        c = pm.make(1, 4, 1, 128, 64, "bf16", "bf16", [130])
        page, slot = int(c.page_table[0, 2]), 2
        c.pages[0, page, :, :, slot:] = bad
        c.set_lengths(ints([90]))
        q = queries(40, 4, 128, "bf16")
        check_attend(c, q, [90], [40])


def test_attend_large_and_small_scores():
    # scores in the thousands, and queries of zeros
    torch, pm = T(), M()
    for typ, kv in (("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "int4")):
        c = pm.make(1, 4, 2, 128, 64, typ, kv, [400])
        c.set_lengths(ints([100]))
        q = queries(300, 4, 128, typ)
        q[::3] *= 100
        q[1::3] = 0
        check_attend(c, q, [100], [300])


def test_attend_is_the_same_from_call_to_call():
    torch = T()
    for d, kv in ((64, "bf16"), (128, "bf16"), (256, "int4")):
        c, q, (out, lse) = attended(5, 12, 4, d, 32, "bf16", kv, [0, 500, 20, 3, 0], [300, 7, 64, 0, 1], bias=True)
        for _ in range(5):
            junk = torch.full((1 << 22,), math.nan, device="cuda")     # other values in what is handed out next
            del junk
            o2, l2 = c.attend(0, q, tok_offsets=offsets([300, 7, 64, 0, 1]), return_lse=True)
            assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_attend_captured_and_on_streams():
    torch, pm = T(), M()
    held, new = [600, 20, 0], [40, 100, 5]
    c = pm.make(3, 8, 2, 128, 32, "bf16", "bf16", [640, 120, 5], softcap=25.0)
    c.set_lengths(ints(held))
    offs = offsets(new)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graphs, ins, outs = [], [], []
    for s in streams:
        gr, qi = torch.cuda.CUDAGraph(), torch.zeros(145, 8, 128, device="cuda").bfloat16()
        with torch.cuda.graph(gr, stream=s):
            outs.append(c.attend(0, qi, tok_offsets=offs, return_lse=True))
        graphs.append(gr), ins.append(qi)
    for rep in range(5):
        for i, qi in enumerate(ins):
            qi.copy_(queries(145, 8, 128, "bf16", 10 * rep + i))
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for got, qi in zip(outs, ins):
            check_attend(c, qi, held, new, got=got)
    q = queries(145, 8, 128, "bf16")
    s = streams[0]
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
        got = c.attend(0, q, tok_offsets=offs, return_lse=True, stream=stream)
        rows = c.read(0, 145, tok_offsets=offs, stream=stream)
        junk = [torch.full_like(q, 3.0) for _ in range(20)]
        torch.cuda.synchronize()
        check_attend(c, q, held, new, got=got)
        assert len(junk) == 20 and torch.equal(rows, c.read(0, 145, tok_offsets=offs))
    assert c.device_error() == 0


# ---- one token: caps, biases, 4-bit pages -----------------------------------------------------------

def check_decode(c, q, lengths, layer=0, got=None):
    torch, pm = T(), M()
    out, lse = c.decode(layer, q, return_lse=True) if got is None else got
    for r, n in enumerate(lengths):
        pos = torch.tensor([n - 1], device="cuda")
        want, wl, tol, tl = pm.attend(c, layer, r, q[r:r + 1], pos, n, one=True)
        pm.within(lse[r:r + 1], wl, tl, f"lse of request {r} (length {n})")
        pm.within(out[r:r + 1], want, tol, f"out of request {r} (length {n})")
    return out, lse


def decoded(R, hq, hk, d, page, typ, kv, lengths, seed=0, bias=False, **kw):
    pm = M()
    c = pm.make(R, hq, hk, d, page, typ, kv, lengths, seed=seed, slopes=pm.slopes_of(hq) if bias else None, **kw)
    c.set_lengths(ints(lengths))
    check_decode(c, queries(R, hq, d, typ, seed), lengths)
    assert c.device_error() == 0


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 130, 1000]


@pytest.mark.parametrize("typ", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq, hk, page", [(4, 4, 16), (8, 1, 64), (12, 4, 32), (32, 2, 128), (40, 1, 256), (7, 1, 16)])
def test_decode_4bit_lengths_and_heads(typ, d, hq, hk, page):
    decoded(len(LENGTHS), hq, hk, d, page, typ, "int4", LENGTHS, seed=d + hq)


@pytest.mark.parametrize("typ, kv", KINDS)
@pytest.mark.parametrize("d, hq, hk", [(64, 6, 2), (128, 16, 1), (256, 10, 1)])
@pytest.mark.parametrize("window, softcap, bias", [(0, 30.0, False), (0, 0.0, True), (100, 2.0, True), (37, 1000.0, False)])
def test_decode_scores(typ, kv, d, hq, hk, window, softcap, bias):
    decoded(8, hq, hk, d, 16, typ, kv, [0, 1, 40, 777, 5, 2049, 64, 300], window=window, softcap=softcap, bias=bias, seed=d)


@pytest.mark.parametrize("lengths", [[30000], [9001, 3], [1] * 200, [0] * 5, [700] * 20])
@pytest.mark.parametrize("d, hq, hk, window", [(128, 8, 1, 0), (64, 8, 2, 0), (256, 12, 1, 300), (128, 32, 8, 5000)])
def test_decode_4bit_splits(lengths, d, hq, hk, window):
    decoded(len(lengths), hq, hk, d, 64, "bf16", "int4", lengths, window=window)


def test_decode_4bit_skips_bad_pages_and_rows():
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import hs
    for d in (64, 128, 256):
        c = pm.make(3, 4, 1, d, 32, "fp16", "int4", [200, 70, 33], extra_pages=1)
        c.set_lengths(ints([200, 70, 33]))
        c.page_table[0, 2] = -5
        c.page_table[1, 2] = c.n_pages + 3
        q = queries(3, 4, d, "fp16")
        check_decode(c, q, [200, 70, 33])
        assert c.device_error() == hs.HS_DEVERR_PAGE
        c.lengths[1] = 10 ** 6
        c.next_lengths.copy_(c.lengths)
        out, lse = c.decode(0, q, return_lse=True, req_ids=ints([9, 1, 2]))
        assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
        assert c.device_error() == hs.HS_DEVERR_PAGE | hs.HS_DEVERR_CAPACITY | hs.HS_DEVERR_REQ_RANGE


def test_4bit_pages_take_every_code_and_scale():
    # all sixteen codes, the smallest, the largest and negative scales: what rows hold is what is attended and read
    torch, pm = T(), M()
    for d in (64, 128, 256):
        c = pm.make(1, 2, 1, d, 16, "bf16", "int4", [0], extra_pages=2, power_of_two=True)
        g = torch.Generator(device="cuda").manual_seed(d)
        raw = torch.randint(0, 256, c.pages.shape, generator=g, device="cuda").to(torch.uint8)
        s = raw[..., 8 * d:]
        s[(s & 0x7F) == 0x7F] = 0x31                      # no NaN
        c.pages.copy_(raw)
        c.set_lengths(ints([0]))
        rows, _ = pm.rows_of(c, 0, 0, 29)
        got = c.read(0, 29, tok_offsets=ints([0, 29]))
        assert torch.equal(got, rows.to(torch.bfloat16))  # codes of 4 bits, scales of 4 and a power of two: exact in bf16
        c.set_lengths(ints([29]))
        # scores of up to 256 * 448 * 8 * ...: small queries
        q = (queries(1, 2, d, "bf16").float() * 1e-4).bfloat16()
        check_decode(c, q, [29])


# ---- rows into 4-bit pages, and back ------------------------------------------------------------------

def test_append_4bit_codes():
    # unrotated rows: the very bytes of the formula, and nothing else changed
    torch, pm = T(), M()
    for typ, d, hk, page in (("bf16", 128, 8, 64), ("fp16", 64, 3, 16), ("bf16", 256, 2, 32), ("fp16", 128, 1, 256)):
        held, new = [0, 17, 5, 300, 40], [20, 0, 1, 333, 64]
        c = pm.make(5, hk, hk, d, page, typ, "int4", held, extra_pages=25)
        c.set_lengths(ints(held))
        n = sum(new)
        g = torch.Generator(device="cuda").manual_seed(d)
        kv = torch.randn(n, 2 * hk * d, generator=g, device="cuda") * torch.rand(n, 1, generator=g, device="cuda").mul(6).exp()
        kv[3] = 0
        kv[5, :16] = 1e-6
        kv[7] *= 1e3
        kv = kv.to(pm.DT[typ])
        k, v = kv[:, :hk * d].view(n, hk, d), kv[:, hk * d:].view(n, hk, d)
        want = c.pages.clone()
        pos = torch.cat([torch.arange(a, a + b, device="cuda") for a, b in zip(held, new)])
        req = torch.cat([torch.full((b,), r, device="cuda") for r, b in enumerate(new)])
        rows = torch.stack([k, v], 1)
        pm.put4(want[0], c.page_table[req, pos // page], pos % page, *pm.quantise(rows, c.kv_scale[0]))
        c.append(0, k, v, tok_offsets=offsets(new))
        assert torch.equal(c.pages, want)
        assert c.next_lengths.tolist() == [a + b for a, b in zip(held, new)] and c.lengths.tolist() == held
        got = c.read(0, n, tok_offsets=offsets(new))
        assert got.shape == (n, 2, hk, d)
        exact = torch.stack([pm.rows_of(c, 0, r, held[r] + new[r])[0][p] for r, p in zip(req.tolist()[::7], pos.tolist()[::7])])
        # two products in 32 bits, one rounding
        pm.within(got[::7], exact, (plain.HALF_STEP[pm.DT[typ]] + 2.0 ** -22) * exact.abs() + plain.TINY[pm.DT[typ]], "read")
        assert c.device_error() == 0


def test_append_4bit_nan_infinity_and_border_values():
    torch, pm = T(), M()
    d, hk = 64, 1
    c = pm.make(1, 1, hk, d, 16, "bf16", "int4", [0], extra_pages=1, power_of_two=True)
    ks = c.kv_scale[0].clone()
    x = torch.randn(6, hk, d, device="cuda").bfloat16()
    x[0, 0, 3] = math.nan
    x[1, 0, 20] = math.inf
    x[2, 0, 40] = -math.inf
    x[3, 0] = 1e30
    x[4, 0] = 1e-30
    x[5, 0, :16] = torch.arange(-8, 8, device="cuda").bfloat16()
    c.append(0, x, x, tok_offsets=ints([0, 6]))
    for w in (0, 1):
        got = c.read(0, 6, tok_offsets=ints([0, 6]))[:, w, 0].float() / ks[w, 0]
        assert torch.isnan(got[0, :16]).all() and not torch.isnan(got[0, 16:]).any()
        assert got[1, 20] == 448 * 7 and got[2, 40] == -448 * 7 and torch.isfinite(got[1:3]).all()
        assert (got[3] == 448 * 7).all() and (got[4] == 0).all()
    code, scale = pm.quantise(torch.stack([x, x], 1), ks)
    want = c.pages.clone()
    pm.put4(want[0], c.page_table[0, :1].expand(6), torch.arange(6, device="cuda"), code, scale)
    assert torch.equal(c.pages, want)


def quiet_rows(n, hk, d, typ, ks, seed):
    """Rows [n, 2, hk, d] whose blocks' largest |x / kv_scale| lies between 2^-12 and 2^-2: near every border of the
    subnormal scales k 2^-9 and of the first normal ones, and anywhere between; ks a power of two."""
    torch, pm = T(), M()
    g = torch.Generator(device="cuda").manual_seed(seed + 41)
    blocks = n * 2 * hk * (d // 16)
    # s changes at amax / 7 = (k + 1/2) 2^-9, codes of the largest element at |x| = 7.5 s: there, one step of the type up and down
    k = torch.arange(0, 16, device="cuda", dtype=torch.float64)
    edges = torch.cat([7 * (2 * k + 1) * 2.0 ** -10, 7.5 * k[1:] * 2.0 ** -9, 7 * k[1:] * 2.0 ** -9])
    step = 1 + 2 * pm.HALF_STEP[pm.DT[typ]]
    edges = torch.cat([edges, edges * step, edges / step])
    top = torch.exp2(torch.rand(blocks, generator=g, device="cuda", dtype=torch.float64) * 10 - 12)
    near = torch.randint(0, 2 * len(edges), (blocks,), generator=g, device="cuda")
    top = torch.where(near < len(edges), edges[near.clamp(max=len(edges) - 1)], top)
    x = torch.rand(blocks, 16, generator=g, device="cuda", dtype=torch.float64) * 2 - 1
    x[:, 0], x[:, 1] = 1, -1
    x = x.gather(1, torch.rand(blocks, 16, generator=g, device="cuda").argsort(1))
    x[::2] *= torch.randint(0, 2, (len(x[::2]), 1), generator=g, device="cuda") * 2 - 1
    return ((x * top[:, None]).view(n, 2, hk, d) * ks.double()[None, :, :, None]).to(pm.DT[typ])


@pytest.mark.parametrize("typ, d, hk, page", [("bf16", 64, 3, 16), ("bf16", 128, 8, 64), ("bf16", 256, 2, 32), ("fp16", 64, 1, 256),
                                              ("fp16", 128, 2, 16), ("fp16", 256, 3, 128)])
def test_append_4bit_codes_of_quiet_rows(typ, d, hk, page):
    # below 2^-6 the scales of blocks are multiples of 2^-9, whose rounding leaves quotients of up to 10.5: codes stay in +-7
    torch, pm = T(), M()
    held, new = [0, 17, 5], [40, 333, 64]
    c = pm.make(3, hk, hk, d, page, typ, "int4", held, extra_pages=25, power_of_two=True)
    c.set_lengths(ints(held))
    n = sum(new)
    rows = quiet_rows(n, hk, d, typ, c.kv_scale[0], d + hk)
    pos = torch.cat([torch.arange(a, a + b, device="cuda") for a, b in zip(held, new)])
    req = torch.cat([torch.full((b,), r, device="cuda") for r, b in enumerate(new)])
    want = c.pages.clone()
    code, scale = pm.quantise(rows, c.kv_scale[0])
    assert len(scale.unique()) > 15 and int(scale.min()) == 0 and int(code.min()) == 1 and int(code.max()) == 15
    pm.put4(want[0], c.page_table[req, pos // page], pos % page, code, scale)
    c.append(0, rows[:, 0], rows[:, 1], tok_offsets=offsets(new))
    assert torch.equal(c.pages, want)
    # and what a reader gets: a code of 4 bits, scales of 4 and a power of two, exact in either type
    value = (code.double() - 8) * scale.contiguous().view(torch.float8_e4m3fn).double() * c.kv_scale[0].double()[None, :, :, None]
    assert torch.equal(c.read(0, n, tok_offsets=offsets(new)).double(), value)
    assert c.device_error() == 0


@pytest.mark.parametrize("sigma", [0.005, 0.01, 0.02, 0.03, 0.05, 0.2])
@pytest.mark.parametrize("d, rot, inter", [(64, 64, False), (128, 128, True), (256, 64, False)])
def test_append_4bit_quiet_rows_rotated(sigma, d, rot, inter):
    # normal rows under kv_scale 1: every element within half a step of its block's scale, or, where a scale rounded down
    # leaves the largest above 7 of it, within what is cut off there
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import PagedKVCache, Rotary
    hk, n = 4, 300
    R = Rotary(rot, interleaved=inter)
    c = PagedKVCache(n_layers=1, n_pages=20, page_size=16, max_requests=1, max_pages=20, h_q=hk, h_kv=hk, d=d, kv_dtype="int4",
                     kv_scale=torch.ones(1, 2, hk, device="cuda"), rotary=R)
    c.reserve(0, n)
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = ((torch.randn(n, hk, d, generator=g, device="cuda") * sigma).bfloat16() for _ in range(3))
    offs, pos = ints([0, n]), torch.arange(n, device="cuda")
    c.append(0, k, v, q=q, tok_offsets=offs)
    kr, tol = plain.rotate(k, pos.int(), plain.frequencies(rot), 1.0, inter)
    got, _ = pm.rows_of(c, 0, 0, n)
    units = c.pages[0][c.page_table[0, pos // 16].long(), :, :, 0]
    for w, (x, t) in enumerate(((kr, tol), (v.double(), torch.zeros_like(tol)))):
        _, at = (p[w].to(x.device) for p in pm.places(d))
        s = units[:, w].gather(-1, at[pos % 16][:, None, :].expand(n, hk, d)).contiguous().view(torch.float8_e4m3fn).double()
        wide = lambda y: y.unflatten(-1, (-1, 16)).amax(-1, keepdim=True).expand(n, hk, d // 16, 16).flatten(-2)   # noqa: E731
        top, slack = wide(x.abs()), wide(t + 2.0 ** -22 * x.abs())
        # the scale: half a step of e4m3, relative where it is normal, of 2^-9 below
        assert ((s - top / 7).abs() <= (top / 7 * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 2.0 ** -20) + slack).all()
        off = (got[:, w] - x).abs()
        assert (off <= torch.maximum(s * (0.5 + 2.0 ** -20), top - 7 * s) + 2 * slack).all()
        assert (got[:, w] * x >= -(slack * s)).all()                  # no element's sign turns
    assert torch.equal(c.read(0, n, tok_offsets=offs, starts=ints([0])).double(), got)
    assert c.device_error() == 0


@pytest.mark.parametrize("d, rot, inter, shift", [(128, 128, False, 0), (64, 32, True, 0), (256, 64, False, 0), (128, 128, True, 1),
                                                  (64, 6, False, 1), (256, 250, False, 0)])
def test_append_4bit_rotated(d, rot, inter, shift):
    # rotated keys within half a step of their block's scale; queries as Rotary.apply turns them; slices of one projection,
    # of any alignment
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import Rotary
    hq, hk, held, new = 6, 2, [3, 100, 0], [70, 1, 33]
    R = Rotary(rot, interleaved=inter)
    c = pm.make(3, hq, hk, d, 32, "bf16", "int4", held, extra_pages=4, rotary=R)
    c.set_lengths(ints(held))
    n = sum(new)
    wide = torch.randn(n * (hq + 2 * hk) * d + 8, device="cuda").bfloat16()[shift:shift + n * (hq + 2 * hk) * d].view(n, -1)
    q, k, v = (wide[:, a * d:b * d].view(n, b - a, d) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    pos = torch.cat([torch.arange(a, a + b, device="cuda") for a, b in zip(held, new)]).int()
    qr = c.append(0, k, v, q=q, tok_offsets=offsets(new))
    assert torch.equal(qr, R.apply(pos, q))
    req = torch.cat([torch.full((b,), r, device="cuda") for r, b in enumerate(new)])
    freqs = plain.frequencies(rot)
    kr, tol = plain.rotate(k, pos, freqs, 1.0, inter)
    page, slot = c.page_table[req, pos // 32].long(), (pos % 32).long()
    units = c.pages[0][page, :, :, slot // 16]
    for w, (x, t) in enumerate(((kr, tol), (v.double(), torch.zeros_like(tol)))):
        x, t = x / c.kv_scale[0, w].double()[None, :, None], t / c.kv_scale[0, w].double()[None, :, None]
        t = t + 2.0 ** -22 * x.abs()
        got = pm.values4(units[:, w], w, d)[torch.arange(n, device="cuda"), :, slot % 16]
        _, at = (p[w].to(x.device) for p in pm.places(d))
        sb = units[:, w].gather(-1, at[slot % 16][:, None, :].expand(n, hk, d))
        s = sb.contiguous().view(torch.float8_e4m3fn).double()
        top = x.abs().unflatten(-1, (-1, 16)).amax(-1, keepdim=True).expand(n, hk, d // 16, 16).flatten(-2)
        slack = t.unflatten(-1, (-1, 16)).amax(-1, keepdim=True).expand(n, hk, d // 16, 16).flatten(-2)
        assert ((s - top / 7).abs() <= (2.0 ** -4 + 2.0 ** -20) * (top / 7 + slack) + 2.0 ** -10 + slack).all()
        # half a step of the block's scale, and of the quotient's rounding; a clamped code is within that too
        assert ((got - x).abs() <= s * (0.5 + 2.0 ** -20) + slack).all()
    again = q.contiguous()
    assert c.append(0, k, v, q=again, q_out=again, tok_offsets=offsets(new)) is again and torch.equal(again, qr)
    assert c.device_error() == 0


def test_append_4bit_skips_bad_requests_pages_and_offsets():
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import hs
    c = pm.make(4, 2, 2, 64, 16, "fp16", "int4", [5, 20, 0, 30], extra_pages=1)
    c.set_lengths(ints([5, 20, 0, 30]))
    before = c.pages.clone()
    x = torch.randn(12, 2, 64, device="cuda").half()
    c.page_table[0, 0] = -1
    c.lengths[1] = -3
    c.append(0, x, x, req_ids=ints([0, 1, 55, 3]), tok_offsets=ints([1, 4, 7, 9, 11]))
    assert c.device_error() == hs.HS_DEVERR_PAGE | hs.HS_DEVERR_CAPACITY | hs.HS_DEVERR_REQ_RANGE
    want = before.clone()
    rows = torch.stack([x, x], 1)[9:11]
    pos = torch.tensor([30, 31], device="cuda")
    pm.put4(want[0], c.page_table[3, pos // 16], pos % 16, *pm.quantise(rows, c.kv_scale[0]))
    assert torch.equal(c.pages, want)
    assert c.next_lengths.tolist() == [8, -3, 0, 32]
    # no tokens at all: next lengths only
    c._error.zero_()
    c.set_lengths(ints([5, 20, 0, 30]))
    c.next_lengths.fill_(99)
    c.append(0, x[:0], x[:0], tok_offsets=ints([0, 0, 0, 0, 0]))
    assert c.next_lengths.tolist() == [5, 20, 0, 30] and torch.equal(c.pages, want)


@pytest.mark.parametrize("typ, kv", KINDS)
@pytest.mark.parametrize("d, hk, page", [(64, 3, 16), (128, 8, 64), (256, 1, 256)])
def test_read(typ, kv, d, hk, page):
    torch, pm = T(), M()
    totals = [40, 0, 333, 16]
    c = pm.make(4, hk, hk, d, page, typ, kv, totals)
    starts, n = ints([7, 0, 100, 15]), [33, 0, 200, 1]
    out = torch.full((240, 2 * hk + 1, d), 7.0, device="cuda").to(pm.DT[typ])
    rows = out[:, :2 * hk].unflatten(1, (2, hk))
    assert c.read(0, 240, tok_offsets=offsets(n, 3), starts=starts, out=rows) is rows
    at = 3
    for r, m in enumerate(n):
        if m:
            want, _ = pm.rows_of(c, 0, r, totals[r])
            want = want[int(starts[r]):][:m]
            # code times scales: two products in 32 bits, then one rounding
            tol = plain.HALF_STEP[pm.DT[typ]] * want.abs() * (1 + 2.0 ** -20) + plain.TINY[pm.DT[typ]] + 2.0 ** -22 * want.abs()
            pm.within(rows[at:at + m], want, tol if c.kv_scale is not None else torch.zeros_like(tol), f"rows of request {r}")
        at += m
    assert (out[:3] == 7).all() and (out[at:] == 7).all() and (out[:, 2 * hk] == 7).all()
    # the step's new rows by default; the same number for each request
    c.set_lengths(ints([0, 0, 5, 0]))
    assert torch.equal(c.read(0, 6, req_ids=ints([2, 3])), torch.cat([c.read(0, 3, req_ids=ints([r])) for r in (2, 3)]))
    assert c.device_error() == 0


def test_read_bad_requests_and_pages():
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import hs
    for kv in ("bf16", "int4"):
        c = pm.make(3, 2, 2, 64, 16, "bf16", kv, [40, 40, 40])
        c.page_table[1, 1] = 10 ** 6
        got = c.read(0, 60, req_ids=ints([0, 99, 1]), starts=ints([0, 5, 0]))
        assert c.device_error() == hs.HS_DEVERR_REQ_RANGE | hs.HS_DEVERR_PAGE
        assert (got[20:40] == 0).all() and not (got[:20] == 0).all(-1).any()
        # (request 1 starts at 5: its second page from row 11 on)
        assert (got[51:] == 0).all() and not (got[40:51] == 0).all(-1).any()


def test_a_request_moves_to_the_two_tier_cache():
    # what outgrows HBM: rows read out of 4-bit pages, flattened, are what the two-tier cache takes
    import numpy as np
    torch, pm = T(), M()
    from oracle import sparse_attention
    from tests.harness import MAX_ABS, REL_L2, attention_error
    from tiered_kv_cache_int8_gb300 import HiSparseCache
    n, hq, hk, d = 60, 8, 2, 128
    c = pm.make(2, hq, hk, d, 16, "bf16", "int4", [5, n])
    rows = c.read(0, n, req_ids=ints([1]), starts=ints([0, 0])).view(1, n, 2 * hk * d)
    two = HiSparseCache(n_layers=1, max_requests=1, max_context=64, h_q=hq, h_kv=hk, d_qk=d, d_v=d, d_idx=64, top_k=64, hot_slots=64)
    two.append(0, rows, torch.randint(-127, 128, (1, n, 64), device="cuda", dtype=torch.int8))
    q = torch.randn(1, hq, d, device="cuda").bfloat16()
    out = two.decode_layer(0, torch.zeros(1, 64, dtype=torch.int8, device="cuda"), q)
    as_bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)   # noqa: E731
    ref = sparse_attention(as_bits(q[0]), as_bits(rows[0]), h_kv=hk, d_qk=d, d_v=d, v_offset=hk * d)
    ma, rel = attention_error(as_bits(out[0]), ref)
    assert ma <= MAX_ABS and rel <= REL_L2
    two.close()


# ---- offsets of more than 32 bits -------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int4"])
def test_pages_behind_32_bits(kv):
    # a pool of more than 2^32 bytes (of 16-bit pages: elements), a request on its last pages and one on its first
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    hq, hk, d, page, n_pages = 16, 8, 128, 64, 66000
    ks = None if kv == "bf16" else torch.full((1, 2, hk), 0.01 if kv == "e4m3" else 0.5, device="cuda")
    c = PagedKVCache(n_layers=1, n_pages=n_pages, page_size=page, max_requests=2, max_pages=16, h_q=hq, h_kv=hk, d=d,
                     kv_dtype=pm.DT.get(kv, kv), kv_scale=ks)
    assert c.pages.numel() > 1 << 32
    held, new = [700, 90], [70, 40]
    c.page_table[0, :14] = torch.arange(n_pages - 1, n_pages - 15, -1, device="cuda", dtype=torch.int32)
    c.page_table[1, :4] = torch.arange(4, device="cuda", dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(5)
    for r in range(2):
        pm.fill(c, 0, r, 0, held[r], g)
    c.set_lengths(ints(held))
    k, v = (torch.randn(110, hk, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    c.append(0, k, v, tok_offsets=offsets(new))
    check_attend(c, queries(110, hq, d, "bf16"), held, new)
    c.commit()
    check_decode(c, queries(2, hq, d, "bf16", 1), [770, 130])
    rows = c.read(0, 70, req_ids=ints([0]), starts=ints([700, 0]))
    want, _ = pm.rows_of(c, 0, 0, 770)
    pm.within(rows, want[700:], pm.HALF_STEP[torch.bfloat16] * want[700:].abs() * (1 + 2.0 ** -12), "rows")
    # what was stored is what was given: to its own type, to e4m3's half a step (and the type's), to half of a 4-bit one
    x = torch.stack([k[:70], v[:70]], 1).double()
    amax = x.unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, -1, 16).flatten(-2)
    tol = {"bf16": 0 * x, "e4m3": x.abs() * 2.0 ** -4 + 0.01 * 2.0 ** -10, "int4": amax * (0.5 / 7) * 1.0625 + 1e-6}[kv]
    pm.within(want[700:], x, tol * (1 + 2.0 ** -10), "stored rows")
    assert c.device_error() == 0


def test_rows_of_a_call_behind_31_bits():
    # more than 2^31 elements of queries, outputs and rows read: 4096 requests that share their pages
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    R, n, hq, hk, d, page = 4096, 130, 64, 16, 64, 64
    c = PagedKVCache(n_layers=1, n_pages=8, page_size=page, max_requests=R, max_pages=4, h_q=hq, h_kv=hk, d=d)
    c.page_table.copy_(torch.arange(4, device="cuda", dtype=torch.int32).expand(R, 4))
    pm.fill(c, 0, 0, 0, 170, torch.Generator(device="cuda").manual_seed(3))
    c.set_lengths(torch.full((R,), 40, dtype=torch.int32, device="cuda"))
    q = queries(n, hq, d, "bf16").repeat(R, 1, 1)
    assert q.numel() > 1 << 31
    ends = torch.arange(R + 1, dtype=torch.int32, device="cuda") * n
    out, lse = c.attend(0, q, tok_offsets=ends, return_lse=True)
    pos = torch.arange(40, 40 + n, device="cuda")
    for r in (0, R // 2, R - 1):
        rows = slice(r * n, (r + 1) * n)
        want, wl, tol, tl = pm.attend(c, 0, r, q[rows], pos, 40 + n)
        pm.within(lse[rows], wl, tl, f"lse of request {r}")
        pm.within(out[rows], want, tol, f"out of request {r}")
    del q, out, lse
    rows = c.read(0, R * 170 * 2, tok_offsets=torch.arange(R, 2 * R + 1, dtype=torch.int32, device="cuda") * 170,
                  starts=torch.zeros(R, dtype=torch.int32, device="cuda"))
    want, _ = pm.rows_of(c, 0, 0, 170)
    assert rows.numel() > 1 << 31
    for r in (R, 2 * R - 1):                       # (rows before the first offset are nobody's)
        assert torch.equal(rows[r * 170:(r + 1) * 170].double(), want)
    del rows
    # rows far apart
    big = torch.empty(10, 1 << 28, dtype=torch.bfloat16, device="cuda")
    few = c.read(0, 10, req_ids=ints([R - 1]), starts=torch.zeros(R, dtype=torch.int32, device="cuda"),
                 out=big[:, :2 * hk * d].unflatten(1, (2, hk, d)))
    assert torch.equal(few.double(), want[:10])
    q = big[:, 4096:4096 + hq * d].unflatten(1, (hq, d))
    q.copy_(queries(10, hq, d, "bf16", 7))
    got = c.attend(0, q, req_ids=ints([R - 1]), return_lse=True)
    check_attend(c, q, [40] * R, [10], ids=[R - 1], got=got)
    assert c.device_error() == 0


@pytest.mark.parametrize("kv", ["bf16", "int4"])
@pytest.mark.parametrize("window", [0, 1000])
def test_the_last_positions_of_the_longest_request(kv, window):
    # 2^22 positions, most of them on one page that they share
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    N, page, hq, d = 1 << 22, 256, 4, 64
    c = PagedKVCache(n_layers=1, n_pages=12, page_size=page, max_requests=1, max_pages=N // page, h_q=hq, h_kv=1, d=d, window=window,
                     kv_dtype=pm.DT.get(kv, kv), kv_scale=None if kv == "bf16" else torch.full((1, 2, 1), 0.5, device="cuda"),
                     softcap=20.0, slopes=pm.slopes_of(hq))
    c.page_table.zero_()
    c.page_table[0, -10:] = torch.arange(1, 11, device="cuda", dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(6)
    pm.fill(c, 0, 0, 0, page, g)
    pm.fill(c, 0, 0, N - 10 * page, N, g)
    c.set_lengths(ints([N - 40]))
    check_attend(c, queries(40, hq, d, "bf16"), [N - 40], [40])
    c.set_lengths(ints([N]))
    check_decode(c, queries(1, hq, d, "bf16", 1), [N])
    assert c.device_error() == 0


# ---- together -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("typ, kv, d", [("bf16", "bf16", 128), ("fp16", "int4", 64), ("bf16", "int4", 128), ("bf16", "e4m3", 256)])
def test_a_model_serves(typ, kv, d):
    # prompts of different lengths, drafted tokens, then single tokens, over two layers
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import PagedKVCache, Rotary
    L, R, hq, hk, page = 2, 3, 8, 2, 16
    ks = None if kv == typ else torch.full((L, 2, hk), 0.02 if kv == "e4m3" else 0.7, device="cuda")
    c = PagedKVCache(n_layers=L, n_pages=60, page_size=page, max_requests=R, max_pages=16, h_q=hq, h_kv=hk, d=d, dtype=pm.DT[typ],
                     kv_dtype=pm.DT.get(kv, kv), rotary=Rotary(d, base=500000.0), kv_scale=ks, softcap=30.0, slopes=pm.slopes_of(hq))
    c.pages.view(torch.uint8).fill_(0x7F)
    held = [0, 0, 0]
    for new in ([19, 1, 140], [4, 4, 4], [1, 1, 1], [0, 70, 0], [1, 1, 1]):
        n = sum(new)
        for r in range(R):
            c.reserve(r, held[r] + new[r])
        for layer in range(L):
            q, k, v = (torch.randn(n, h, d, device="cuda").to(pm.DT[typ]) for h in (hq, hk, hk))
            q = c.append(layer, k, v, q=q, tok_offsets=offsets(new))
            if new == [1, 1, 1]:
                check_decode(c, q, [h + 1 for h in held], layer)
            check_attend(c, q, held, new, layer=layer)
        held = [a + b for a, b in zip(held, new)]
        c.commit()
        assert c.lengths.tolist() == held
    assert c.device_error() == 0


def test_a_captured_step_with_drafted_tokens():
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import Rotary
    held = [100, 0]
    c = pm.make(2, 4, 2, 64, 16, "bf16", "int4", held, extra_pages=4, rotary=Rotary(64))
    c.set_lengths(ints(held))
    q, k, v = (torch.randn(6, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    offs = offsets([3, 3])
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        qr = c.append(0, k, v, q=q, tok_offsets=offs)
        got = c.attend(0, qr, tok_offsets=offs, return_lse=True)
        rows = c.read(0, 6, tok_offsets=offs)
    for _ in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn_like(x))
        gr.replay()
        torch.cuda.synchronize()
        check_attend(c, qr, held, [3, 3], got=got)
        assert torch.equal(rows, c.read(0, 6, tok_offsets=offs))
        c.commit()
        held = [n + 3 for n in held]
        assert c.lengths.tolist() == held


# ---- refusals ----------------------------------------------------------------------------------------------

def test_refusals_of_the_binding():
    torch, pm = T(), M()
    from tiered_kv_cache_int8_gb300 import HsError, PagedKVCache
    kw = dict(n_layers=1, n_pages=4, page_size=16, max_requests=2, max_pages=2, h_q=4, h_kv=2, d=64)
    ks = torch.ones(1, 2, 2, device="cuda")
    for bad in (dict(kv_dtype="int8"), dict(dtype="int4"), dict(kv_dtype="int4", kv_scale=ks[0]), dict(slopes=torch.ones(3, device="cuda")),
                dict(slopes=torch.ones(4)), dict(slopes=torch.ones(4, device="cuda").half()),
                dict(kv_dtype="int4", kv_scale=ks, pages=torch.zeros(1, 4, 2, 2, 16, 64, device="cuda").bfloat16())):
        with pytest.raises(ValueError):
            PagedKVCache(**{**kw, **bad})
    for bad in (dict(kv_dtype="int4"), dict(softcap=-1.0), dict(softcap=math.inf), dict(softcap=1e-9), dict(softcap=math.nan)):
        with pytest.raises(HsError):
            PagedKVCache(**{**kw, **bad})
    c = PagedKVCache(**kw, kv_dtype="int4", kv_scale=ks, softcap=5.0, slopes=torch.ones(4, device="cuda"))
    assert c.pages.shape == (1, 4, 2, 2, 1, 576) and c.pages.dtype == torch.uint8
    q = torch.zeros(4, 4, 64, device="cuda").bfloat16()
    two = ints([0, 2, 4])
    for call in (lambda: c.attend(0, q.half(), tok_offsets=two), lambda: c.attend(0, q[:, :2], tok_offsets=two),
                 lambda: c.attend(0, q, tok_offsets=two.long()), lambda: c.attend(0, q, tok_offsets=two, prefix=ints([0])),
                 lambda: c.attend(0, q, tok_offsets=two, lengths=ints([0])), lambda: c.attend(0, q, tok_offsets=two, out=q[:3]),
                 lambda: c.attend(0, q, tok_offsets=two, out=q.transpose(0, 1)), lambda: c.attend(0, q.cpu(), tok_offsets=two),
                 lambda: c.read(0, -1), lambda: c.read(0, 4, tok_offsets=two, out=q), lambda: c.read(0, 4, tok_offsets=two.cpu()),
                 lambda: c.read(0, 4, tok_offsets=two, starts=ints([1])), lambda: setattr(c, "slopes", None)):
        with pytest.raises((ValueError, AttributeError)):
            call()
    for call in (lambda: c.attend(0, q), lambda: c.attend(1, q, tok_offsets=two), lambda: c.read(1, 4, tok_offsets=two),
                 lambda: c.attend(0, torch.zeros(4, 4, 65, device="cuda").bfloat16()[:, :, 1:], tok_offsets=two),
                 lambda: c.read(0, 3, req_ids=ints([0, 1]))):
        with pytest.raises(HsError):
            call()
    assert c.attend(0, q[:0], tok_offsets=ints([0, 0, 0])).shape == (0, 4, 64)
    assert c.read(0, 0, tok_offsets=ints([0, 0, 0])).shape == (0, 2, 2, 64)
