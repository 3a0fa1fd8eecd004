"""Rotary tables and the refusals of the rotary and paged-cache entry points: no GPU needed."""
import ctypes
import math

import pytest

from tests.paged_plain import frequencies, magnitude


@pytest.fixture(scope="module")
def L():
    from tiered_kv_cache_int8_gb300.build import build
    build()
    from tiered_kv_cache_int8_gb300 import hs
    return hs.lib()


def table(L, rot, base=10000.0, scaling=None, inv_freq=None, mag=0.0):
    from tiered_kv_cache_int8_gb300 import hs
    kinds = {None: 0, "linear": 1, "ntk": 2, "by_parts": 3}
    s = dict(scaling or {})
    cfg = hs.HsRotaryConfig(base, s.get("factor", 1.0), s.get("original_context", 0.0), s.get("low", 1.0),
                            s.get("high", 32.0), mag, rot, kinds.get(s.get("kind"), 9))
    n = max(1, rot // 2)
    turns, m = (ctypes.c_uint64 * n)(), ctypes.c_float(-1)
    f = None if inv_freq is None else (ctypes.c_double * n)(*inv_freq)
    rc = L.hs_rotary_table(ctypes.byref(cfg), f, turns, ctypes.byref(m))
    return rc, list(turns), m.value


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 1024])
@pytest.mark.parametrize("scaling", [None, {"kind": "linear", "factor": 4.0}, {"kind": "ntk", "factor": 8.0},
                                     {"kind": "by_parts", "factor": 8.0, "original_context": 8192.0},
                                     {"kind": "by_parts", "factor": 32.0, "original_context": 100.0, "low": 0.5,
                                      "high": 4.0}])
def test_rotary_table_follows_the_formulas(L, rot, scaling):
    if rot == 2 and (scaling or {}).get("kind") == "ntk":
        assert table(L, rot, scaling=scaling)[0] == -2
        return
    rc, turns, mag = table(L, rot, base=500000.0, scaling=scaling)
    assert rc == 0
    want = frequencies(rot, 500000.0, scaling)
    for t, f in zip(turns, want):
        # an entry is off by a few roundings of a double (pow, division) and one step of 2^-64
        assert abs(t / 2.0 ** 64 - (f / (2 * math.pi)) % 1.0) <= 8 * 2.0 ** -53 * f / (2 * math.pi) + 2.0 ** -63
    assert mag == pytest.approx(magnitude(scaling), rel=2.0 ** -23)


def test_rotary_table_of_given_frequencies(L):
    given = [7.5, 1.0, 1e-3, 0.0]
    rc, turns, mag = table(L, 8, base=0.0, inv_freq=given, mag=1.25)
    assert rc == 0 and mag == 1.25
    for t, f in zip(turns, given):
        # the fraction of a turn of 7.5 radians loses the whole turn exactly
        assert abs(t / 2.0 ** 64 - (f / (2 * math.pi)) % 1.0) <= 2.0 ** -51


@pytest.mark.parametrize("kw", [
    dict(rot=3), dict(rot=0), dict(rot=-2), dict(rot=1026), dict(rot=8, base=1.0), dict(rot=8, base=math.inf),
    dict(rot=8, base=math.nan), dict(rot=8, mag=-1.0), dict(rot=8, mag=math.nan),
    dict(rot=8, scaling={"kind": "linear", "factor": 0.5}), dict(rot=8, scaling={"kind": "linear", "factor": math.nan}),
    dict(rot=8, scaling={"kind": "other"}), dict(rot=8, scaling={"kind": "by_parts", "factor": 2.0}),
    dict(rot=8, scaling={"kind": "by_parts", "factor": 2.0, "original_context": 64.0, "low": 2.0, "high": 2.0}),
    dict(rot=4, inv_freq=[1.0, -1.0]), dict(rot=4, inv_freq=[math.inf, 1.0]),
])
def test_rotary_table_refusals(L, kw):
    assert table(L, **kw)[0] == -2
    assert L.hs_last_error(None).decode().startswith("hs_rotary_table:")


def heads(data=4096, ts=256, hs_=64, h=4):
    from tiered_kv_cache_int8_gb300 import hs
    return hs.HsHeads(data, ts, hs_, h, 0)


@pytest.mark.parametrize("what", ["type", "d_small", "d_large", "n_tok", "views", "null_rot", "null_in", "table", "odd_table",
                                  "rot_large", "rot_odd", "layout", "transpose", "magnitude", "positions", "odd_positions",
                                  "null_data", "heads", "negative", "odd_data", "overlapping_out", "broadcast_out",
                                  "other_heads", "in_out_overlap"])
def test_rotary_apply_refusals(L, what):
    # addresses are never followed: every call is refused before any device work
    from tiered_kv_cache_int8_gb300 import hs
    rot = hs.HsRotary(4096, 64, 0, 0, 1.0)
    a = dict(type=hs.HS_BF16, d=64, n=5, pos=4096, views=1)
    i, o = heads(), heads(data=1 << 20)
    if what == "type": a["type"] = hs.HS_E4M3
    if what == "d_small": a["d"] = 1
    if what == "d_large": a["d"] = 1026
    if what == "n_tok": a["n"] = -1
    if what == "views": a["views"] = 3
    if what == "table": rot.turns = None
    if what == "odd_table": rot.turns = 4100
    if what == "rot_large": rot.rot_dim = 66
    if what == "rot_odd": rot.rot_dim = 7
    if what == "layout": rot.interleaved = 2
    if what == "transpose": rot.transpose = -1
    if what == "magnitude": rot.magnitude = math.nan
    if what == "positions": a["pos"] = None
    if what == "odd_positions": a["pos"] = 4098
    if what == "null_data": i.data = None
    if what == "heads": i.heads = o.heads = 0
    if what == "negative": i.token_stride = -256
    if what == "odd_data": i.data = 4097
    if what == "overlapping_out": o.head_stride = 63
    if what == "broadcast_out": o.token_stride = 0
    if what == "other_heads": o.heads = 3
    if what == "in_out_overlap": o.data = i.data + 128
    rc = L.hs_rotary_apply(None if what == "null_rot" else ctypes.byref(rot), a["type"], a["d"], a["n"], a["pos"], a["views"],
                           None if what == "null_in" else ctypes.byref(i), ctypes.byref(o), 0, None)
    assert rc == hs.HS_ERR_INVALID
    assert L.hs_last_error(None).decode().startswith("hs_rotary_apply:")


def test_rotary_apply_of_no_tokens_is_a_no_op(L):
    from tiered_kv_cache_int8_gb300 import hs
    rot = hs.HsRotary(4096, 64, 0, 0, 1.0)
    i, o = heads(), heads()
    assert L.hs_rotary_apply(ctypes.byref(rot), hs.HS_FP32, 64, 0, None, 1, ctypes.byref(i), ctypes.byref(o), 0, None) == 0


def paged_cfg(**over):
    from tiered_kv_cache_int8_gb300 import hs
    base = dict(n_layers=2, n_pages=10, page_size=64, max_requests=8, max_pages=5, h_q=8, h_kv=2, d=128, type=hs.HS_BF16,
                page_type=hs.HS_BF16, window=0, device=0, softmax_scale=0.0)
    base.update(over)
    return hs.HsPagedConfig(**base)


def create(L, pages=4096, scale=None, err=4096, **over):
    h = ctypes.c_void_p()
    return L.hs_paged_create(ctypes.byref(paged_cfg(**over)), pages, scale, err, ctypes.byref(h)), h


@pytest.mark.parametrize("over", [
    dict(n_layers=0), dict(n_pages=0), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(max_requests=0),
    dict(max_requests=4097), dict(max_pages=0), dict(max_pages=1 << 17), dict(d=96), dict(d=0), dict(h_kv=0), dict(h_q=9),
    dict(h_q=1), dict(type=2, page_type=2), dict(type=3, page_type=3), dict(page_type=1), dict(window=-1),
    dict(softmax_scale=-1.0), dict(softmax_scale=math.inf), dict(n_pages=1 << 24, page_size=256, h_kv=2),
])
def test_paged_create_refuses_configurations(L, over):
    rc, h = create(L, **over)
    assert rc == -2 and not h
    assert L.hs_last_error(None).decode().startswith("hs_paged_create:")


@pytest.mark.parametrize("kw", [dict(pages=None), dict(pages=4104), dict(scale=4096), dict(page_type=3), dict(err=None),
                                dict(err=4097), dict(page_type=3, scale=4098)])
def test_paged_create_refuses_buffers(L, kw):
    rc, h = create(L, **kw)
    assert rc == -1 and not h


def test_paged_create_holds_host_memory_only(L):
    rc, h = create(L)
    assert rc == 0 and h
    L.hs_paged_destroy(h)
    L.hs_paged_destroy(None)
    assert L.hs_paged_create(None, 4096, None, 4096, ctypes.byref(h)) == -1


@pytest.mark.parametrize("what", ["handle", "layer", "n_req", "n_tok", "uneven", "table", "lengths", "odd", "next_is_lengths",
                                  "next_overlaps", "q_alone", "q_without_rot", "rot_large", "transposed", "k", "k_heads",
                                  "q_heads", "v_null", "q_out_overlap", "k_odd"])
def test_paged_append_refusals(L, what):
    from tiered_kv_cache_int8_gb300 import hs
    _, h = create(L)
    rot = hs.HsRotary(4096, 128, 0, 0, 1.0)
    q, qo = heads(1 << 20, 1024, 128, 8), heads(1 << 24, 1024, 128, 8)
    k, v = heads(1 << 26, 256, 128, 2), heads(1 << 27, 256, 128, 2)
    a = dict(h=h, layer=0, n_req=4, n_tok=8, table=4096, lengths=1 << 14, nxt=1 << 15, ids=None)
    R = ctypes.byref
    q_, qo_, k_, v_, r_ = R(q), R(qo), R(k), R(v), R(rot)
    if what == "handle": a["h"] = None
    if what == "layer": a["layer"] = 2
    if what == "n_req": a["n_req"] = 9
    if what == "n_tok": a["n_tok"] = -4
    if what == "uneven": a["n_tok"] = 9
    if what == "table": a["table"] = None
    if what == "lengths": a["lengths"] = None
    if what == "odd": a["ids"] = 4097
    if what == "next_is_lengths": a["nxt"] = a["lengths"]
    if what == "next_overlaps": a["nxt"] = a["lengths"] + 28
    if what == "q_alone": qo_ = None
    if what == "q_without_rot": r_ = None
    if what == "rot_large": rot.rot_dim = 130
    if what == "transposed": rot.transpose = 1
    if what == "k": k_ = None
    if what == "k_heads": k.heads = 3
    if what == "q_heads": q.heads = qo.heads = 4
    if what == "v_null": v.data = None
    if what == "q_out_overlap": qo.data = q.data + 16
    if what == "k_odd": k.data = k.data + 1
    rc = L.hs_paged_append(a["h"], a["layer"], a["n_req"], a["ids"], a["n_tok"], None, a["table"], a["lengths"], a["nxt"], r_,
                           q_, qo_, k_, v_, None)
    assert rc == hs.HS_ERR_INVALID
    assert L.hs_last_error(None).decode().startswith("hs_paged_append:")
    L.hs_paged_destroy(h)


@pytest.mark.parametrize("what", ["handle", "layer", "n_req", "table", "lengths", "q", "out", "ws", "odd_out", "odd_ws", "odd_lse",
                                  "q_heads", "q_rows", "q_data"])
def test_paged_decode_refusals(L, what):
    from tiered_kv_cache_int8_gb300 import hs
    _, h = create(L)
    q = heads(1 << 20, 1024, 128, 8)
    a = dict(h=h, layer=1, n_req=3, table=4096, lengths=4096, out=4096, lse=None, ws=4096)
    if what == "handle": a["h"] = None
    if what == "layer": a["layer"] = -1
    if what == "n_req": a["n_req"] = -1
    if what == "table": a["table"] = None
    if what == "lengths": a["lengths"] = None
    if what == "out": a["out"] = None
    if what == "ws": a["ws"] = None
    if what == "odd_out": a["out"] = 4104
    if what == "odd_ws": a["ws"] = 4096 + 128
    if what == "odd_lse": a["lse"] = 4098
    if what == "q_heads": q.heads = 4
    if what == "q_rows": q.token_stride = 1025
    if what == "q_data": q.data = q.data + 2
    rc = L.hs_paged_decode(a["h"], a["layer"], a["n_req"], None, a["table"], a["lengths"],
                           None if what == "q" else ctypes.byref(q), a["out"], a["lse"], a["ws"], None)
    assert rc == hs.HS_ERR_INVALID
    assert L.hs_last_error(None).decode().startswith("hs_paged_decode:")
    L.hs_paged_destroy(h)


def test_calls_of_no_requests_are_no_ops(L):
    _, h = create(L)
    assert L.hs_paged_append(h, 0, 0, None, 0, None, None, None, None, None, None, None, None, None, None) == 0
    assert L.hs_paged_decode(h, 0, 0, None, None, None, None, None, None, None, None) == 0
    L.hs_paged_destroy(h)


@pytest.mark.parametrize("struct, cls", [("hs_heads", "HsHeads"), ("hs_rotary_config", "HsRotaryConfig"), ("hs_rotary", "HsRotary"),
                                         ("hs_paged_config", "HsPagedConfig")])
def test_binding_structs_follow_the_header(struct, cls):
    import os
    import re
    from tests.conftest import ROOT
    from tiered_kv_cache_int8_gb300 import hs
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hs.h")).read(), flags=re.S)
    body = re.search(r"typedef struct " + struct + r"\s*\{(.*?)\}\s*" + struct + r"_t;", text, flags=re.S).group(1)
    ctype = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float, "double": ctypes.c_double,
             "void*": ctypes.c_void_p, "const uint64_t*": ctypes.c_void_p}
    want = [(m[1], ctype[m[0]]) for m in re.findall(r"(const uint64_t\*|void\*|int32_t|int64_t|float|double)\s+(\w+)\s*;", body)]
    assert list(getattr(hs, cls)._fields_) == want


@pytest.mark.parametrize("n, ts, h, hs_, taken", [
    (1 + (1 << 24), 1 << 40, 4, 64, False),        # 2^64 elements, what wraps around to none
    (1 + (1 << 30), 1 << 33, 4, 64, False), ((1 << 31) - 1, 1 << 40, 1, 0, False), (2, 256, 4096, 1 << 40, False),
    (2, 1 << 40, 66, 1 << 40, False), (65, 1 << 40, 4, 64, True), (66, 1 << 40, 4, 64, False), (1, 1 << 40, 65, 1 << 40, True)])
@pytest.mark.parametrize("which", ["in", "out"])
def test_views_beyond_64_bits_are_refused(L, n, ts, h, hs_, taken, which):
    # device -1: a call whose arguments pass stops at the device, with another code
    from tiered_kv_cache_int8_gb300 import hs
    rot = hs.HsRotary(4096, 64, 0, 0, 1.0)
    far, near = heads(1 << 50, ts, hs_, h), heads(1 << 12, 64 * h, 64, h)
    if not taken:
        near.data = far.data + 2 * ts              # on far's second row, or apart from it only modulo 2^64
    i, o = (far, near) if which == "in" else (near, far)
    rc = L.hs_rotary_apply(ctypes.byref(rot), hs.HS_BF16, 64, n, 4096, 1, ctypes.byref(i), ctypes.byref(o), -1, None)
    if taken:
        assert rc == hs.HS_ERR_CUDA
    else:
        assert rc == hs.HS_ERR_INVALID
        assert "within 2^46" in L.hs_last_error(None).decode()
