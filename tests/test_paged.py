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


def elements(view, n, d):
    return {view.data // 2 + t * view.token_stride + h * view.head_stride + i
            for t in range(n) for h in range(view.heads) for i in range(d)}


def apply_two(L, ins, outs, n, d=8):
    # device -1: a call whose arguments pass stops at the device, with another code than a refusal's
    from tiered_kv_cache_int8_gb300 import hs
    rot = hs.HsRotary(4096, d, 0, 0, 1.0)
    rc = L.hs_rotary_apply(ctypes.byref(rot), hs.HS_BF16, d, n, 4096, len(ins), (hs.HsHeads * len(ins))(*ins),
                           (hs.HsHeads * len(outs))(*outs), -1, None)
    assert rc in (hs.HS_ERR_INVALID, hs.HS_ERR_CUDA)
    return rc == hs.HS_ERR_CUDA


@pytest.mark.parametrize("what", ["two_outputs", "swapped", "out0_in1", "out1_in0", "one_input_in_place", "one_row", "shifted"])
def test_rotary_apply_refuses_outputs_over_the_other_view(L, what):
    a, b = heads(1 << 12, 32, 8, 4), heads(1 << 16, 32, 8, 4)
    x, y = heads(1 << 20, 32, 8, 4), heads(1 << 24, 32, 8, 4)
    assert apply_two(L, (a, b), (x, y), 5) and apply_two(L, (a, b), (a, b), 5) and apply_two(L, (a, a), (x, y), 5)
    ins, outs = {"two_outputs": ((a, b), (x, x)), "swapped": ((a, b), (b, a)), "out0_in1": ((a, b), (b, y)),
                 "out1_in0": ((a, b), (x, a)), "one_input_in_place": ((a, a), (a, y)),
                 "one_row": ((a, heads(1 << 16, 32, 8, 1)), (x, heads(x.data + 4 * 64 + 3 * 16, 32, 8, 1))),   # x's last
                 "shifted": ((a, b), (x, heads(x.data + 8, 32, 8, 4)))}[what]
    assert not apply_two(L, ins, outs, 5)
    assert "overlaps the other" in L.hs_last_error(None).decode()


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("layout", ["projection", "interleaved", "heads_first", "alternate_rows", "heads_first_interleaved"])
def test_rotary_apply_takes_slices_of_one_buffer_in_place(L, n, layout):
    # queries of 4 heads of 8 elements and keys of 4 (projection: of 2)
    q, k = {"projection": (heads(4096, 64, 8, 4), heads(4096 + 64, 64, 8, 2)),
            "interleaved": (heads(4096, 96, 24, 4), heads(4096 + 16, 96, 24, 4)),         # [n][heads][q, k, v][8]
            "heads_first": (heads(4096, 8, 8 * n, 4), heads(4096 + 64 * n, 8, 8 * n, 4)),  # [heads][n][8]
            "alternate_rows": (heads(4096, 64, 8, 4), heads(4096 + 64, 64, 8, 4)),
            "heads_first_interleaved": (heads(4096, 24, 24 * n, 4), heads(4096 + 32, 24, 24 * n, 4))}[layout]
    assert not elements(q, n, 8) & elements(k, n, 8)
    assert apply_two(L, (q, k), (q, k), n) and apply_two(L, (k, q), (k, q), n)
    away = heads(1 << 20, 32, 8, 4), heads(1 << 24, 8 * k.heads, 8, k.heads)
    assert apply_two(L, (q, k), away, n) and apply_two(L, (q, k), (q, away[1]), n)


def test_no_overlap_passes(L):
    # small views of any strides: a call that passes has outputs apart from each other and from the other input
    import random
    rng = random.Random(7)
    passed = 0
    for _ in range(4000):
        n = rng.randint(1, 4)
        out = [heads(4096 + 2 * rng.randint(0, 160), rng.choice([0, 4, 8, 12, 16, 24, 40, 48]), rng.choice([0, 4, 8, 12, 20, 32, 48, 96]),
                     rng.randint(1, 3)) for _ in range(2)]
        other = heads(4096 + 2 * rng.randint(0, 160), rng.choice([0, 4, 8, 12, 24, 40]), rng.choice([0, 4, 12, 32]), out[1].heads)
        ins = [out[0], out[1] if rng.random() < 0.5 else other]
        if apply_two(L, ins, out, n, d=4):
            passed += 1
            sets = [elements(v, n, 4) for v in (out[0], out[1], ins[1])]
            assert all(len(s) == n * v.heads * 4 for s, v in zip(sets, out))
            assert not sets[0] & sets[1] and not sets[0] & sets[2]
            if ins[1] is not out[1]:
                assert not sets[1] & sets[2]
    assert passed > 100


@pytest.mark.parametrize("what", ["fine", "k", "v", "k_row", "v_slice"])
def test_paged_append_refuses_queries_over_new_rows(L, what):
    from tiered_kv_cache_int8_gb300 import hs
    _, h = create(L, device=-1)
    rot = hs.HsRotary(4096, 128, 0, 0, 1.0)
    # slices of one projection, rotated in place: 8 + 2 + 2 heads of 128
    q, k, v = heads(1 << 20, 1536, 128, 8), heads((1 << 20) + 2048, 1536, 128, 2), heads((1 << 20) + 2560, 1536, 128, 2)
    qo = q
    if what == "k": qo = heads(k.data, 1024, 128, 8)
    if what == "v": qo = heads(1 << 24, 1024, 128, 8); v = heads(1 << 24, 256, 128, 2)
    if what == "k_row": qo = heads(1 << 24, 1024, 128, 8); k = heads((1 << 24) + 7 * 2048 + 1792, 1536, 128, 2)
    if what == "v_slice": qo = heads(q.data + 256, 1536, 128, 8); q = heads(1 << 24, 1024, 128, 8); v = heads((1 << 20) + 256, 1536, 128, 2)
    R = ctypes.byref
    rc = L.hs_paged_append(h, 0, 4, None, 8, None, 4096, 1 << 14, 1 << 15, R(rot), R(q), R(qo), R(k), R(v), None)
    assert rc == (hs.HS_ERR_CUDA if what == "fine" else hs.HS_ERR_INVALID)
    if what != "fine":
        assert "overlaps" in L.hs_last_error(None).decode()
    L.hs_paged_destroy(h)


@pytest.mark.parametrize("name", ["pages", "kv_scale", "page_table", "lengths", "next_lengths"])
def test_the_cache_keeps_its_tensors(name):
    # the library holds their addresses, or is given them unchecked: another tensor in their place would be misread
    import torch
    from tiered_kv_cache_int8_gb300 import PagedKVCache
    cache = object.__new__(PagedKVCache)
    cache._h = None
    held = torch.ones(3, dtype=torch.int32)
    setattr(cache, "_" + name, held)
    with pytest.raises(AttributeError):
        setattr(cache, name, torch.zeros(1, dtype=torch.int64))
    setattr(cache, name, getattr(cache, name).__iadd__(1))      # as `cache.lengths += 1` does
    assert getattr(cache, name) is held and held.tolist() == [2, 2, 2]


def test_a_stream_of_another_device_is_refused():
    import types
    import torch
    from tiered_kv_cache_int8_gb300 import paged
    other = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError):
        paged._on_stream(other, torch.device("cuda", 0), (), lambda: pytest.fail("the call was made"))
