"""What hs_paged_set_scores, hs_paged_attend, hs_paged_read and 4-bit pages refuse, through the C
ABI and without a GPU, and the layout of 4-bit units."""
import ctypes
import math

import pytest

from tests.test_paged import L, create, heads  # noqa: F401 (L: a fixture)


@pytest.mark.parametrize("kw, rc", [
    (dict(page_type=4), -1), (dict(page_type=4, scale=4098), -1), (dict(page_type=5), -2), (dict(page_type=4, type=4, scale=4096), -2),
    (dict(page_type=4, scale=4096, pages=4104), -1), (dict(page_type=4, scale=4096), 0),
])
def test_create_with_4bit_pages(L, kw, rc):   # noqa: F811
    got, h = create(L, **kw)
    assert got == rc and bool(h) == (rc == 0)
    L.hs_paged_destroy(h)


@pytest.mark.parametrize("cap, slopes, rc", [(-1.0, None, -2), (math.inf, None, -2), (math.nan, None, -2), (1e-5, None, -2),
                                             (2e6, None, -2), (0.0, 4098, -1), (0.0, None, 0), (50.0, 4096, 0)])
def test_set_scores_refusals(L, cap, slopes, rc):   # noqa: F811
    _, h = create(L)
    assert L.hs_paged_set_scores(h, cap, slopes) == rc
    if rc:
        assert L.hs_last_error(None).decode().startswith("hs_paged_set_scores:")
    assert L.hs_paged_set_scores(None, 0.0, None) == -1
    L.hs_paged_destroy(h)


@pytest.mark.parametrize("what", ["handle", "layer", "n_req", "n_tok", "uneven", "table", "lengths", "q", "out", "ws", "odd_ids",
                                  "odd_prefix", "odd_lse", "odd_out", "odd_ws", "q_heads", "q_rows", "q_data", "overlap", "rows"])
def test_attend_refusals(L, what):   # noqa: F811
    from tiered_kv_cache_int8_gb300 import hs
    _, h = create(L)
    q = heads(1 << 20, 1024, 128, 8)
    a = dict(h=h, layer=1, n_req=4, ids=None, n=8, table=4096, lengths=8192, prefix=None, out=1 << 24, lse=None, ws=4096)
    if what == "handle": a["h"] = None
    if what == "layer": a["layer"] = 2
    if what == "n_req": a["n_req"] = 9
    if what == "n_tok": a["n"] = -8
    if what == "uneven": a["n"] = 9
    if what == "table": a["table"] = None
    if what == "lengths": a["lengths"] = None
    if what == "out": a["out"] = None
    if what == "ws": a["ws"] = None
    if what == "odd_ids": a["ids"] = 4097
    if what == "odd_prefix": a["prefix"] = 4098
    if what == "odd_lse": a["lse"] = 4097
    if what == "odd_out": a["out"] += 8
    if what == "odd_ws": a["ws"] += 128
    if what == "q_heads": q.heads = 4
    if what == "q_rows": q.token_stride = 1025
    if what == "q_data": q.data += 2
    if what == "overlap": a["out"] = q.data + 2048
    if what == "rows":
        a["n"] = 1 << 30
        q.token_stride = 0
    rc = L.hs_paged_attend(a["h"], a["layer"], a["n_req"], a["ids"], a["n"], None, a["table"], a["lengths"], a["prefix"],
                           None if what == "q" else ctypes.byref(q), a["out"], a["lse"], a["ws"], None)
    assert rc == hs.HS_ERR_INVALID
    assert L.hs_last_error(None).decode().startswith("hs_paged_attend:")
    L.hs_paged_destroy(h)


@pytest.mark.parametrize("what", ["handle", "layer", "n_req", "n_tok", "uneven", "table", "starts", "out", "odd_ids", "odd_starts",
                                  "odd_out", "stride", "odd_stride", "far"])
def test_read_refusals(L, what):   # noqa: F811
    from tiered_kv_cache_int8_gb300 import hs
    _, h = create(L)
    a = dict(h=h, layer=1, n_req=4, ids=None, n=8, table=4096, starts=8192, out=1 << 24, stride=512)
    if what == "handle": a["h"] = None
    if what == "layer": a["layer"] = -1
    if what == "n_req": a["n_req"] = -1
    if what == "n_tok": a["n"] = -8
    if what == "uneven": a["n"] = 7
    if what == "table": a["table"] = None
    if what == "starts": a["starts"] = None
    if what == "out": a["out"] = None
    if what == "odd_ids": a["ids"] = 4097
    if what == "odd_starts": a["starts"] = 8194
    if what == "odd_out": a["out"] += 8
    if what == "stride": a["stride"] = 504
    if what == "odd_stride": a["stride"] = 516
    if what == "far": a["stride"] = (1 << 40) + 8
    rc = L.hs_paged_read(a["h"], a["layer"], a["n_req"], a["ids"], a["n"], None, a["table"], a["starts"], a["out"], a["stride"], None)
    assert rc == hs.HS_ERR_INVALID
    assert L.hs_last_error(None).decode().startswith("hs_paged_read:")
    L.hs_paged_destroy(h)


def test_calls_of_nothing_are_no_ops(L):   # noqa: F811
    _, h = create(L)
    for n_req in (0, 3):
        assert L.hs_paged_attend(h, 0, n_req, None, 0, None, None, None, None, None, None, None, None, None) == 0
        assert L.hs_paged_read(h, 0, n_req, None, 0, None, None, None, None, 0, None) == 0
    assert L.hs_paged_attend_workspace_bytes(None) == 0
    L.hs_paged_destroy(h)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_4bit_units_fill_their_bytes(d):
    # of 16 rows: every half byte of the first 8 d holds one code, every byte of the last d one block's scale
    from tests.paged_more import places
    code, scale = places(d)
    for w in (0, 1):
        assert sorted(code[w].flatten().tolist()) == sorted(list(range(8 * d)) * 2)
        assert sorted(set(scale[w].flatten().tolist())) == list(range(8 * d, 9 * d))
        at = {}
        for i in range(16):
            for e in range(d):
                at.setdefault(int(scale[w, i, e]), set()).add((i, e // 16))
        assert all(len(x) == 1 for x in at.values())
