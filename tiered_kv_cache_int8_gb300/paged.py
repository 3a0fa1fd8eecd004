"""Rotary positions and the paged cache: the binding of hs_rotary_* and hs_paged_*
(include/hs.h states what they compute).

Every step runs in the library's CUDA kernels.  Calls run on the current stream
of their device, or on ``stream``; a call's own outputs and workspace are
allocated on that stream.  ``ValueError`` for tensors of a wrong shape, type or
device, ``HsError`` for what the library refuses.
"""
from __future__ import annotations

import ctypes

import torch

from .hs import (HS_BF16, HS_E4M3, HS_ERR_DEVICE, HS_FP16, HS_FP32, HS_OK, HS_ROTARY_BY_PARTS, HS_ROTARY_LINEAR,
                 HS_ROTARY_NTK, HS_ROTARY_PLAIN, HsError, HsHeads, HsPagedConfig, HsRotary, HsRotaryConfig, lib)

TYPES = {torch.bfloat16: HS_BF16, torch.float16: HS_FP16, torch.float32: HS_FP32, torch.float8_e4m3fn: HS_E4M3}
_ROTATED = {torch.bfloat16: HS_BF16, torch.float16: HS_FP16, torch.float32: HS_FP32}
_VIEWS = (None, HsHeads * 1, HsHeads * 2)
SCALINGS = {"linear": HS_ROTARY_LINEAR, "ntk": HS_ROTARY_NTK, "by_parts": HS_ROTARY_BY_PARTS}


_MOST = (1 << 31) - 1
_HEADS_BYTES = ctypes.sizeof(HsHeads)


def _check(rc: int):
    if rc != HS_OK:
        raise HsError(rc, lib().hs_last_error(None).decode())


def _need(ok: bool, why: str):
    if not ok:
        raise ValueError(why)


def _heads(name: str, x, device, dtype, d: int | None = None, heads: int | None = None) -> HsHeads:
    """The [tokens, heads, d] view of a tensor whose last dimension is dense."""
    if x.dim() != 3 or x.device != device or x.dtype != dtype:
        raise ValueError(f"{name} must be [tokens, heads, d] {dtype} on {device}, not {list(x.shape)} {x.dtype} on {x.device}")
    _, h, e = x.shape
    if (d is not None and e != d) or (heads is not None and h != heads):
        raise ValueError(f"{name} must be [tokens, {heads}, {d}], not {list(x.shape)}")
    ts, hs, es = x.stride()
    if es != 1 and e > 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    return HsHeads(x.data_ptr(), ts, hs, h, 0)


def _dense(x, shape) -> HsHeads:
    """The view of a new tensor of that shape."""
    _, h, d = shape
    return HsHeads(x.data_ptr(), h * d, d, h, 0)


def _ints(name: str, x, device, n: int):
    if x.dtype != torch.int32 or x.device != device or x.shape != (n,) or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [{n}] on {device}, "
                         f"not {list(x.shape)} {x.dtype} on {x.device}")
    return x.data_ptr()


# the current stream's handle, without building the Stream object where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

def _on_stream(call, stream, device, tensors):
    """call(handle) on a given stream: what it allocates belongs to that stream, and the
    given tensors are marked as used there."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.cuda_stream == _raw_stream(device.index):
        return call(stream.cuda_stream)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


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

        out       : the tensor(s) to write: the inputs themselves (in place) or others
        transpose : the transposed rotation (angles negated): what takes a gradient of
                    the rotated values back; the inverse where magnitude is 1
        """
        k = len(xs)
        if k != 1 and k != 2:
            raise ValueError("apply takes one or two tensors")
        dev, x0, x1 = self.device, xs[0], xs[-1]
        dtype = x0.dtype
        if dtype not in _ROTATED:
            raise ValueError(f"no rotation of {dtype}")
        views = _VIEWS[k](*[_heads("x", x, dev, dtype) for x in xs])
        n, _, d = x0.shape
        if n > _MOST:
            raise ValueError("more than 2^31 - 1 tokens")
        if k == 2 and (x1.shape[0] != n or x1.shape[2] != d):
            raise ValueError("the tensors have different tokens or widths")
        pos = _ints("positions", positions, dev, n)
        if out is None:
            outs = None
        else:
            outs = (out,) if isinstance(out, torch.Tensor) else tuple(out)
            if len(outs) != k or any(o.shape != x.shape for o, x in zip(outs, xs)):
                raise ValueError("out must have the shapes of the inputs")

        def call(raw):
            ys = outs
            if ys is None:
                ys = tuple([torch.empty(x.shape, dtype=dtype, device=dev) for x in xs])
                into = _VIEWS[k](*[_dense(y, x.shape) for x, y in zip(xs, ys)])
            else:
                into = _VIEWS[k](*[_heads("out", y, dev, dtype) for y in ys])
            rc = lib().hs_rotary_apply(self._plan[1 if transpose else 0], _ROTATED[dtype], d, n, pos, k, views, into,
                                       dev.index, raw)
            if rc:
                _check(rc)
            return ys[0] if k == 1 else ys

        if stream is None:
            return call(_raw_stream(dev.index))
        return _on_stream(call, stream, dev, (positions, self._table, *xs, *(outs or ())))


class PagedKVCache:
    """A paged cache of keys and values in HBM, its append and its one-token attention.

    pages      : [n_layers, n_pages, 2, h_kv, page_size, d] (given, or allocated here)
    page_table : int32 [max_requests, max_pages], page ids of each request (-1: none);
                 written by ``reserve`` / ``release``, or by the caller, who then hands
                 out the pages
    lengths    : int32 [max_requests], positions held before the step
    next_lengths : with the tokens that ``append`` stored; ``decode`` attends to these,
                 and ``commit`` makes them the lengths once every layer is through

    Calls that write nothing in common may run at once on different streams.
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
        self.pages, self.kv_scale = pages, kv_scale
        self.page_table = torch.full((max_requests, max_pages), -1, dtype=torch.int32, device=self.device)
        self.lengths = torch.zeros(max_requests, dtype=torch.int32, device=self.device)
        self.next_lengths = torch.zeros(max_requests, dtype=torch.int32, device=self.device)
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

    def _tensors(self):
        """The cache's own tensors that a call uses."""
        table = None if self.rotary is None else self.rotary._table
        return self.pages, self.page_table, self.lengths, self.next_lengths, self.kv_scale, self._error, table

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
        self.page_table[req, len(have):need] = torch.tensor(new, dtype=torch.int32, device=self.device)
        have.extend(new)

    def release(self, req: int):
        """Takes back the pages of ``req``: its table row is cleared and its lengths are 0."""
        _need(0 <= req < self.max_requests, "request out of range")
        self._free.extend(reversed(self._held.pop(req, [])))
        self.page_table[req] = -1
        self.lengths[req] = 0
        self.next_lengths[req] = 0

    def free_pages(self) -> int:
        return len(self._free)

    def set_lengths(self, lengths):
        """Positions held by every request (int32 [max_requests])."""
        self.lengths.copy_(lengths)
        self.next_lengths.copy_(lengths)

    def commit(self):
        """The step is through every layer: its tokens count as held."""
        self.lengths.copy_(self.next_lengths)

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
        """
        dev, dtype, n = self.device, self.dtype, k.shape[0]
        views = _VIEWS[2](_heads("k", k, dev, dtype, self.d, self.h_kv), _heads("v", v, dev, dtype, self.d, self.h_kv))
        if v.shape[0] != n:
            raise ValueError("k and v have different numbers of rows")
        if n > _MOST:
            raise ValueError("more than 2^31 - 1 rows")
        n_req, ids, offs = n, None, None
        if req_ids is not None:
            n_req = req_ids.shape[0]
            ids = _ints("req_ids", req_ids, dev, n_req)
        if tok_offsets is not None:
            if req_ids is None:
                n_req = tok_offsets.shape[0] - 1
            offs = _ints("tok_offsets", tok_offsets, dev, n_req + 1)
        hq = None
        if q is not None:
            if self.rotary is None:
                raise ValueError("q needs a cache with a rotation")
            hq = _heads("q", q, dev, dtype, self.d, self.h_q)
            if q.shape[0] != n or (q_out is not None and q_out.shape != q.shape):
                raise ValueError("q, q_out and k have different rows")
        elif q_out is not None:
            raise ValueError("q_out without q")

        def call(raw):
            out, h_in, h_out = q_out, None, None
            if hq is not None:
                if out is None:
                    out = torch.empty(q.shape, dtype=dtype, device=dev)
                    h_out = ctypes.byref(_dense(out, q.shape))
                else:
                    h_out = ctypes.byref(_heads("q_out", out, dev, dtype, self.d, self.h_q))
                h_in = ctypes.byref(hq)
            rc = lib().hs_paged_append(self._h, layer, n_req, ids, n, offs, self.page_table.data_ptr(),
                                       self.lengths.data_ptr(), self.next_lengths.data_ptr(),
                                       None if self.rotary is None else self.rotary._plan[0], h_in, h_out, views,
                                       ctypes.byref(views, _HEADS_BYTES), raw)
            if rc:
                _check(rc)
            return out

        if stream is None:
            return call(_raw_stream(dev.index))
        return _on_stream(call, stream, dev, (k, v, q, q_out, req_ids, tok_offsets, *self._tensors()))

    def decode(self, layer: int, q, req_ids=None, lengths=None, out=None, return_lse: bool = False, stream=None):
        """Attention of one token per request: q [requests, h_q, d] -> out of its shape
        (and, with return_lse, the float32 [requests, h_q] logarithms of the softmax sums).

        lengths : int32 [max_requests], positions attended to; None: next_lengths
        out     : where to write (q itself, if it is contiguous: in place)
        """
        dev, dtype, n = self.device, self.dtype, q.shape[0]
        hq = ctypes.byref(_heads("q", q, dev, dtype, self.d, self.h_q))
        ids = None if req_ids is None else _ints("req_ids", req_ids, dev, n)
        lens = (self.next_lengths.data_ptr() if lengths is None
                else _ints("lengths", lengths, dev, self.max_requests))
        if out is not None and (out.shape != q.shape or out.dtype != dtype or out.device != dev
                                or not out.is_contiguous()):
            raise ValueError("out must be contiguous, of q's shape, type and device")

        def call(raw):
            o, lse, lse_ptr = out, None, None
            if o is None:
                o = torch.empty(q.shape, dtype=dtype, device=dev)
            if return_lse:
                lse = torch.empty((n, self.h_q), dtype=torch.float32, device=dev)
                lse_ptr = lse.data_ptr()
            ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=dev)
            rc = lib().hs_paged_decode(self._h, layer, n, ids, self.page_table.data_ptr(), lens, hq, o.data_ptr(),
                                       lse_ptr, ws.data_ptr(), raw)
            if rc:
                _check(rc)
            return (o, lse) if return_lse else o

        if stream is None:
            return call(_raw_stream(dev.index))
        return _on_stream(call, stream, dev, (q, req_ids, lengths, out, *self._tensors()))

    # -- errors ----------------------------------------------------------------------
    def device_error(self) -> int:
        """HS_DEVERR_* bits that the calls have set so far (synchronises the device)."""
        w = ctypes.c_uint32(0)
        rc = lib().hs_paged_error(self._h, ctypes.byref(w))
        if rc not in (HS_OK, HS_ERR_DEVICE):
            _check(rc)
        return int(w.value)
