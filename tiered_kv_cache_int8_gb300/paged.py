"""Rotary positions and the paged cache: the binding of hs_rotary_* and hs_paged_*
(include/hs.h states what they compute).

Every step runs in the library's CUDA kernels.  Calls run on the current stream
of their device, or on ``stream``; a call's own outputs and workspace are
allocated on that stream.  ``ValueError`` for tensors of a wrong shape, type or
device, ``HsError`` for what the library refuses.

No call records a gradient: ``append`` and ``decode`` are for serving, what they return
has none; ``Rotary.apply`` refuses tensors that require one while gradients are recorded.
Given outputs count as modified in place (a backward pass that saved one says so).
"""
from __future__ import annotations

import ctypes
import struct

import torch

from .hs import (HS_BF16, HS_E4M3, HS_ERR_DEVICE, HS_FP16, HS_FP32, HS_OK, HS_ROTARY_BY_PARTS, HS_ROTARY_LINEAR,
                 HS_ROTARY_NTK, HS_ROTARY_PLAIN, HsError, HsHeads, HsPagedConfig, HsRotary, HsRotaryConfig, lib)

TYPES = {torch.bfloat16: HS_BF16, torch.float16: HS_FP16, torch.float32: HS_FP32, torch.float8_e4m3fn: HS_E4M3}
_ROTATED = {torch.bfloat16: HS_BF16, torch.float16: HS_FP16, torch.float32: HS_FP32}
# one and two hs_heads_t in a row (packed: a ctypes structure of each costs a small call much of its time)
_ONE, _TWO = struct.Struct("Pqqii").pack, struct.Struct("PqqiiPqqii").pack
assert struct.calcsize("Pqqii") == ctypes.sizeof(HsHeads)
_MOST = (1 << 31) - 1
SCALINGS = {"linear": HS_ROTARY_LINEAR, "ntk": HS_ROTARY_NTK, "by_parts": HS_ROTARY_BY_PARTS}


def _check(rc: int):
    if rc != HS_OK:
        raise HsError(rc, lib().hs_last_error(None).decode())


def _need(ok: bool, why: str):
    if not ok:
        raise ValueError(why)


def _heads(name: str, x, device, dtype, d: int | None = None, heads: int | None = None) -> tuple:
    """hs_heads_t of a [tokens, heads, d] tensor whose last dimension is dense."""
    if x.dim() != 3 or x.device != device or x.dtype != dtype:
        raise ValueError(f"{name} must be [tokens, heads, d] {dtype} on {device}, not {list(x.shape)} {x.dtype} on {x.device}")
    n, h, e = x.shape
    if (d is not None and e != d) or (heads is not None and h != heads) or n > _MOST:
        raise ValueError(f"{name} must be [at most 2^31 - 1 tokens, {heads}, {d}], not {list(x.shape)}")
    ts, hs, es = x.stride()
    if es != 1 and e > 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    return x.data_ptr(), ts, hs, h, 0


def _ints(name: str, x, device, n: int):
    if x.dtype != torch.int32 or x.device != device or x.shape != (n,) or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [{n}] on {device}, "
                         f"not {list(x.shape)} {x.dtype} on {x.device}")
    return x.data_ptr()


# the current stream's handle, without building the Stream object where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_grad_on, _modified = torch.is_grad_enabled, torch.autograd.graph.increment_version


def _on_stream(stream, device, tensors, call):
    """call() with a given stream as the current one: what it allocates belongs to that
    stream, and the given tensors are marked as used there."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, not on {device}")
    if stream.cuda_stream != _raw_stream(device.index):
        for t in tensors:
            if t is not None and t.device == device:     # (others are refused by the call)
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call()


class Rotary:
    """A rotation of the first ``rot_dim`` elements of a head by position * frequency.

    interleaved : pairs (2i, 2i+1) instead of (i, i + rot_dim / 2)
    scaling     : None, or {"kind": "linear" | "ntk" | "by_parts", "factor": f} and, for
                  "by_parts", "original_context", "low" (default 1) and "high" (default 32)
    inv_freq    : frequencies (radians per position, rot_dim / 2 of them) in place of the formulas
    magnitude   : the factor on rotated values; None takes the kind's own
    """

    def __init__(self, rot_dim: int, *, base: float = 10000.0, interleaved: bool = False, scaling: dict | None = None,
                 inv_freq=None, magnitude: float | None = None, device: int = 0):
        kind, sc = HS_ROTARY_PLAIN, dict(scaling or {})
        if sc:
            name = sc.pop("kind", None)
            _need(name in SCALINGS, f"scaling's kind must be one of {sorted(SCALINGS)}")
            kind = SCALINGS[name]
            known = {"factor"} | ({"original_context", "low", "high"} if kind == HS_ROTARY_BY_PARTS else set())
            _need(set(sc) <= known and "factor" in sc and (kind != HS_ROTARY_BY_PARTS or "original_context" in sc),
                  f"scaling of kind {name} takes {sorted(known)}")
        _need(magnitude is None or magnitude > 0, "magnitude must be > 0")
        _need(inv_freq is None or scaling is None, "inv_freq takes the place of the formulas: no scaling beside it")
        cfg = HsRotaryConfig(base, sc.get("factor", 1.0), sc.get("original_context", 0.0), sc.get("low", 1.0),
                             sc.get("high", 32.0), magnitude or 0.0, rot_dim, kind)
        n = max(1, rot_dim // 2)
        freqs = None
        if inv_freq is not None:
            values = [float(f) for f in inv_freq]
            _need(len(values) == n, f"inv_freq must have rot_dim / 2 = {n} entries")
            freqs = (ctypes.c_double * n)(*values)
        turns = (ctypes.c_uint64 * n)()
        mag = ctypes.c_float(0.0)
        _check(lib().hs_rotary_table(ctypes.byref(cfg), freqs, turns, ctypes.byref(mag)))
        self.rot_dim, self.interleaved, self.magnitude = rot_dim, bool(interleaved), float(mag.value)
        self.turns = list(turns)     # as fractions of 2^64 of a turn per position
        self.device = torch.device("cuda", device)
        as_signed = [t - (1 << 64) if t >> 63 else t for t in self.turns]
        self._table = torch.tensor(as_signed, dtype=torch.int64, device=self.device)
        self._plan = tuple(ctypes.byref(HsRotary(self._table.data_ptr(), rot_dim, int(interleaved), t, mag.value))
                           for t in (0, 1))
        # the table's copy is on the stream of the creation; calls may be on any
        torch.cuda.current_stream(self.device).synchronize()

    def apply(self, positions, *xs, out=None, transpose: bool = False, stream=None):
        """Rotates one or two tensors [tokens, heads, d] (a step's queries and keys) of
        the tokens at ``positions`` (int32 [tokens]); returns the rotated tensor(s).

        out       : the tensor(s) to write: the inputs themselves (in place) or others, each
                    apart from the other output and the other input
        transpose : the transposed rotation (angles negated): what takes a gradient of
                    the rotated values back; the inverse where magnitude is 1

        Records no gradient, and refuses tensors that require one while gradients are
        recorded: in a model that trains, call it in an autograd function's forward, and
        transposed in its backward.
        """
        dev, k = self.device, len(xs)
        if stream is not None:
            outs = () if out is None else (out,) if isinstance(out, torch.Tensor) else tuple(out)
            return _on_stream(stream, dev, (positions, self._table, *xs, *outs),
                              lambda: self.apply(positions, *xs, out=out, transpose=transpose))
        if k != 1 and k != 2:
            raise ValueError("apply takes one or two tensors")
        x0 = xs[0]
        if _grad_on() and (x0.requires_grad or (k == 2 and xs[1].requires_grad)):
            raise ValueError("apply records no gradient of its inputs (without one: torch.no_grad(), or detach)")
        dtype, (n, h, d) = x0.dtype, x0.shape if x0.dim() == 3 else (0, 0, 0)
        if dtype not in _ROTATED:
            raise ValueError(f"no rotation of {dtype}")
        views = _heads("x", x0, dev, dtype)
        pos = _ints("positions", positions, dev, n)
        if out is None:
            y0 = torch.empty((n, h, d), dtype=dtype, device=dev)
            into = (y0.data_ptr(), h * d, d, h, 0)
        else:
            ys = (out,) if isinstance(out, torch.Tensor) else tuple(out)
            if len(ys) != k or ys[0].shape != x0.shape:
                raise ValueError("out must be a tensor for each input, of its shape")
            y0, y1 = ys if k == 2 else (*ys, None)
            if _grad_on() and (y0.requires_grad or (k == 2 and y1.requires_grad)):
                raise ValueError("apply records no gradient: out must not require one")
            into = _heads("out", y0, dev, dtype)
        if k == 1:
            views, into = _ONE(*views), _ONE(*into)
        else:
            x1 = xs[1]
            more = _heads("x", x1, dev, dtype, d)
            if x1.shape[0] != n:
                raise ValueError("the tensors have different tokens")
            if out is None:
                h = more[3]
                y1 = torch.empty((n, h, d), dtype=dtype, device=dev)
                into = _TWO(*into, y1.data_ptr(), h * d, d, h, 0)
            else:
                if y1.shape != x1.shape:
                    raise ValueError("out must have the shapes of the inputs")
                into = _TWO(*into, *_heads("out", y1, dev, dtype))
            views = _TWO(*views, *more)
        rc = lib().hs_rotary_apply(self._plan[1 if transpose else 0], _ROTATED[dtype], d, n, pos, k, views, into,
                                   dev.index, _raw_stream(dev.index))
        if rc:
            _check(rc)
        if out is not None:
            _modified(y0)
            if k == 2:
                _modified(y1)
        return y0 if k == 1 else (y0, y1)


def _kept(name: str):
    """A tensor attribute that is changed in place only."""
    def put(self, value):
        if value is not getattr(self, name):     # (what `cache.lengths += 1` puts back is)
            raise AttributeError(f"{name[1:]} is written in place, not exchanged for another tensor")
    return property(lambda self: getattr(self, name), put)


class PagedKVCache:
    """A paged cache of keys and values in HBM, its append and its one-token attention.

    pages      : [n_layers, n_pages, 2, h_kv, page_size, d] (given, or allocated here)
    page_table : int32 [max_requests, max_pages], page ids of each request (-1: none);
                 written by ``reserve`` / ``release``, or by the caller, who then hands
                 out the pages
    lengths    : int32 [max_requests], positions held before the step
    next_lengths : with the tokens that ``append`` stored; ``decode`` attends to these,
                 and ``commit`` makes them the lengths once every layer is through

    These are written in place (``cache.page_table[r] = ids``); the tensors themselves stay
    the cache's.  Lengths are set by ``set_lengths``: what ``decode`` and ``commit`` take are
    the next ones.

    Calls that write nothing in common may run at once on different streams (appends of one
    step to different layers too: the next lengths they write are the same).
    """

    def __init__(self, *, n_layers: int, n_pages: int, page_size: int, max_requests: int, max_pages: int, h_q: int,
                 h_kv: int, d: int, dtype=torch.bfloat16, kv_dtype=None, softmax_scale: float = 0.0, window: int = 0,
                 rotary: Rotary | None = None, kv_scale=None, pages=None, device: int = 0):
        kv_dtype = kv_dtype or dtype
        _need(dtype in TYPES and kv_dtype in TYPES, f"no cache of {kv_dtype} for {dtype}")
        self._h = ctypes.c_void_p()
        self.device = torch.device("cuda", device)
        self.cfg = HsPagedConfig(n_layers, n_pages, page_size, max_requests, max_pages, h_q, h_kv, d, TYPES[dtype],
                                 TYPES[kv_dtype], window, device, softmax_scale, 0)
        self.dtype, self.kv_dtype, self.rotary = dtype, kv_dtype, rotary
        self.n_layers, self.n_pages, self.page_size, self.max_pages = n_layers, n_pages, page_size, max_pages
        self.max_requests, self.h_q, self.h_kv, self.d = max_requests, h_q, h_kv, d
        _need(rotary is None or rotary.device == self.device, "the rotation is on another device")
        shape = (n_layers, n_pages, 2, h_kv, page_size, d)
        if kv_scale is not None:
            _need(tuple(kv_scale.shape) == (n_layers, 2, h_kv) and kv_scale.dtype == torch.float32
                  and kv_scale.device == self.device, f"kv_scale must be float32 [n_layers, 2, h_kv] on {self.device}")
            kv_scale = kv_scale.contiguous()
        if pages is not None:
            _need(tuple(pages.shape) == shape and pages.dtype == kv_dtype and pages.device == self.device
                  and pages.is_contiguous(), f"pages must be a contiguous {kv_dtype} tensor {list(shape)} on {self.device}")
        else:   # what a bad configuration makes of this is refused by the library below
            pages = torch.empty([max(0, s) for s in shape], dtype=kv_dtype, device=self.device)
        self._error = torch.zeros(4, dtype=torch.int32, device=self.device)
        _check(lib().hs_paged_create(ctypes.byref(self.cfg), pages.data_ptr(),
                                     None if kv_scale is None else kv_scale.data_ptr(), self._error.data_ptr(),
                                     ctypes.byref(self._h)))
        self._pages, self._kv_scale = pages, kv_scale
        self._page_table = torch.full((max_requests, max_pages), -1, dtype=torch.int32, device=self.device)
        self._lengths = torch.zeros(max_requests, dtype=torch.int32, device=self.device)
        self._next_lengths = torch.zeros(max_requests, dtype=torch.int32, device=self.device)
        self._ws_bytes = int(lib().hs_paged_workspace_bytes(self._h))
        self._free = list(range(n_pages - 1, -1, -1))
        self._held: dict[int, list[int]] = {}
        torch.cuda.current_stream(self.device).synchronize()

    # -- lifetime --------------------------------------------------------------
    def close(self):
        if self._h:
            lib().hs_paged_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    # The library and the calls keep to these tensors' addresses: others are not put in their place.
    pages, kv_scale, page_table, lengths, next_lengths = map(
        _kept, ("_pages", "_kv_scale", "_page_table", "_lengths", "_next_lengths"))

    def _tensors(self):
        """The cache's own tensors that a call uses."""
        table = None if self.rotary is None else self.rotary._table
        return self._pages, self._page_table, self._lengths, self._next_lengths, self._kv_scale, self._error, table

    # -- pages and lengths -------------------------------------------------------
    def reserve(self, req: int, n_positions: int):
        """Gives request ``req`` pages for ``n_positions`` positions in all (on the current stream)."""
        _need(0 <= req < self.max_requests, "request out of range")
        have = self._held.setdefault(req, [])
        need = -(-n_positions // self.page_size)
        _need(need <= self.max_pages, f"{n_positions} positions are more than max_pages * page_size")
        n = need - len(have)
        if n <= 0:
            return
        if n > len(self._free):
            raise MemoryError(f"{n} pages wanted, {len(self._free)} free")
        new = [self._free.pop() for _ in range(n)]
        self._page_table[req, len(have):need] = torch.tensor(new, dtype=torch.int32, device=self.device)
        have.extend(new)

    def release(self, req: int):
        """Takes back the pages of ``req``: its table row is cleared and its lengths are 0."""
        _need(0 <= req < self.max_requests, "request out of range")
        self._free.extend(reversed(self._held.pop(req, [])))
        self._page_table[req] = -1
        self._lengths[req] = 0
        self._next_lengths[req] = 0

    def free_pages(self) -> int:
        return len(self._free)

    def set_lengths(self, lengths):
        """Positions held by every request (int32 [max_requests]): its lengths and its next ones."""
        self._lengths.copy_(lengths)
        self._next_lengths.copy_(lengths)

    def commit(self):
        """The step is through every layer: its tokens count as held."""
        self._lengths.copy_(self._next_lengths)

    # -- the path ------------------------------------------------------------------
    def append(self, layer: int, k, v, q=None, q_out=None, req_ids=None, tok_offsets=None, stream=None):
        """Stores new keys and values (k, v: [tokens, h_kv, d]), rotated by the cache's
        ``rotary`` at positions lengths[r], lengths[r] + 1, ...; sets next_lengths.

        q           : the step's queries [tokens, h_q, d]; their rotated values are returned
        q_out       : where to write them (q itself: in place)
        tok_offsets : int32 [requests + 1]: request i takes rows tok_offsets[i] .. tok_offsets[i+1]-1;
                      rows outside belong to nobody (their rows of a new q_out are undefined).
                      None: one row per request (with req_ids: the same number for each)
        req_ids     : int32 [requests] distinct ids; None: requests 0, 1, ...

        q_out lies apart from k and v; k, v and q may be slices of one projection.
        """
        dev, dtype = self.device, self.dtype
        if stream is not None:
            return _on_stream(stream, dev, (k, v, q, q_out, req_ids, tok_offsets, *self._tensors()),
                              lambda: self.append(layer, k, v, q, q_out, req_ids, tok_offsets))
        hk, hv = _heads("k", k, dev, dtype, self.d, self.h_kv), _heads("v", v, dev, dtype, self.d, self.h_kv)
        n_req = n = k.shape[0]
        if v.shape[0] != n:
            raise ValueError("k and v have different numbers of rows")
        ids = offs = hq = ho = rot = None
        if req_ids is not None:
            n_req = req_ids.shape[0]
            ids = _ints("req_ids", req_ids, dev, n_req)
        if tok_offsets is not None:
            if req_ids is None:
                n_req = tok_offsets.shape[0] - 1
            offs = _ints("tok_offsets", tok_offsets, dev, n_req + 1)
        if self.rotary is not None:
            rot = self.rotary._plan[0]
        if q is not None:
            if rot is None:
                raise ValueError("q needs a cache with a rotation")
            hq = _ONE(*_heads("q", q, dev, dtype, self.d, self.h_q))
            if q.shape[0] != n or (q_out is not None and q_out.shape != q.shape):
                raise ValueError("q, q_out and k have different rows")
            if q_out is None:
                q_out = torch.empty((n, self.h_q, self.d), dtype=dtype, device=dev)
                ho = _ONE(q_out.data_ptr(), self.h_q * self.d, self.d, self.h_q, 0)
            else:
                ho = _ONE(*_heads("q_out", q_out, dev, dtype, self.d, self.h_q))
                _modified(q_out)
        elif q_out is not None:
            raise ValueError("q_out without q")
        rc = lib().hs_paged_append(self._h, layer, n_req, ids, n, offs, self._page_table.data_ptr(),
                                   self._lengths.data_ptr(), self._next_lengths.data_ptr(), rot, hq, ho, _ONE(*hk),
                                   _ONE(*hv), _raw_stream(dev.index))
        if rc:
            _check(rc)
        return q_out

    def decode(self, layer: int, q, req_ids=None, lengths=None, out=None, return_lse: bool = False, stream=None):
        """Attention of one token per request: q [requests, h_q, d] -> out of its shape
        (and, with return_lse, the float32 [requests, h_q] logarithms of the softmax sums).

        q       : its rows 16-byte aligned; at most max_requests of them
        lengths : int32 [max_requests], positions attended to; None: next_lengths
        out     : where to write (q itself, if it is contiguous: in place)
        """
        dev, dtype = self.device, self.dtype
        if stream is not None:
            return _on_stream(stream, dev, (q, req_ids, lengths, out, *self._tensors()),
                              lambda: self.decode(layer, q, req_ids, lengths, out, return_lse))
        hq = _ONE(*_heads("q", q, dev, dtype, self.d, self.h_q))
        n, lse, lse_ptr = q.shape[0], None, None
        ids = None if req_ids is None else _ints("req_ids", req_ids, dev, n)
        lens = (self._next_lengths.data_ptr() if lengths is None
                else _ints("lengths", lengths, dev, self.max_requests))
        if out is None:
            out = torch.empty((n, self.h_q, self.d), dtype=dtype, device=dev)
        elif out.shape != q.shape or out.dtype != dtype or out.device != dev or not out.is_contiguous():
            raise ValueError("out must be contiguous, of q's shape, type and device")
        else:
            _modified(out)
        if return_lse:
            lse = torch.empty((n, self.h_q), dtype=torch.float32, device=dev)
            lse_ptr = lse.data_ptr()
        ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=dev)
        rc = lib().hs_paged_decode(self._h, layer, n, ids, self._page_table.data_ptr(), lens, hq, out.data_ptr(),
                                   lse_ptr, ws.data_ptr(), _raw_stream(dev.index))
        if rc:
            _check(rc)
        return (out, lse) if return_lse else out

    # -- errors ----------------------------------------------------------------------
    def device_error(self) -> int:
        """HS_DEVERR_* bits that the calls have set so far (synchronises the device)."""
        w = ctypes.c_uint32(0)
        rc = lib().hs_paged_error(self._h, ctypes.byref(w))
        if rc not in (HS_OK, HS_ERR_DEVICE):
            _check(rc)
        return int(w.value)
