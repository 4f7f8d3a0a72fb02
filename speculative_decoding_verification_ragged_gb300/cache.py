"""Binding of the 4-bit paged cache (include/spec_cache.h): append, read,
attend, weights, evict.

Argument marshalling only, like binding.py.  Every function takes
`prepared=True` to return a CacheCall instead of running: its arguments are
marshalled once, each call launches on the then-current stream and returns the
same result tensors, so a serving loop pays one ctypes call per launch.  `stream`
runs a call on another stream than the current one: its inputs have to be ready
there, and the caller waits for that stream before it uses the results elsewhere.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional

import torch

from .binding import SPEC_BF16, SPEC_F32, SpecError, _check, _dev, _on, _tensors, load_library

BLOCK_TOKENS = 32
HEAD_CHANNELS = (64, 128, 256)


class _Cache(C.Structure):
    _fields_ = [("pages", C.c_void_p), ("n_pages", C.c_int64), ("page_tokens", C.c_int32),
                ("H", C.c_int32), ("D", C.c_int32), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("B", C.c_int32), ("max_pages", C.c_int32),
                ("page_table", C.c_void_p)]


class _Rows(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("dtype", C.c_int32),
                ("k_row", C.c_int64), ("k_head", C.c_int64), ("v_row", C.c_int64),
                ("v_head", C.c_int64), ("R_cap", C.c_int32), ("max_rows", C.c_int32),
                ("cu_rows", C.c_void_p), ("start", C.c_void_p), ("score", C.c_void_p),
                ("slot_pos", C.c_void_p), ("pos0", C.c_void_p), ("status", C.c_void_p)]


class _Attention(C.Structure):
    _fields_ = [("q", C.c_void_p), ("dtype", C.c_int32), ("q_row", C.c_int64),
                ("q_head", C.c_int64), ("Hq", C.c_int32), ("R_cap", C.c_int32),
                ("k_max", C.c_int32), ("cu_rows", C.c_void_p), ("len", C.c_void_p),
                ("max_len", C.c_int32), ("scale", C.c_float), ("cap", C.c_float),
                ("slopes", C.c_void_p), ("window", C.c_int32), ("prefix", C.c_int32),
                ("slot_pos", C.c_void_p), ("status", C.c_void_p)]


class _Eviction(C.Structure):
    _fields_ = [("score", C.c_void_p), ("slot_pos", C.c_void_p), ("len", C.c_void_p),
                ("budget", C.c_int32), ("recent", C.c_int32), ("dst_table", C.c_void_p),
                ("dst_pages", C.c_int32), ("kept", C.c_void_p), ("new_len", C.c_void_p),
                ("status", C.c_void_p)]


class PagedCache:
    """A pool of cache pages: a uint8 tensor [n_pages, H, page_tokens / 32, 36 D]
    and the optional per-head scales (float32 [H])."""

    def __init__(self, pages: torch.Tensor, k_scale=None, v_scale=None):
        if pages.dim() != 4 or pages.dtype != torch.uint8:
            raise SpecError("pages must be uint8 [n_pages, H, blocks, 36 D]")
        self.n_pages, self.H, blocks, nbytes = pages.shape
        self.page_tokens, self.D = blocks * BLOCK_TOKENS, nbytes // 36
        if nbytes % 36 or self.D not in HEAD_CHANNELS:
            raise SpecError("a block has 36 D bytes, D one of %s; got %d bytes"
                            % (HEAD_CHANNELS, nbytes))
        for x, what in [(k_scale, "k_scale"), (v_scale, "v_scale")]:
            if x is not None and x.numel() != self.H:
                raise SpecError("%s needs one value per kv head" % what)
        self.pages, self.k_scale, self.v_scale = pages, k_scale, v_scale

    def _tensors(self):
        return self.pages, self.k_scale, self.v_scale

    def _view(self, page_table, B: int) -> _Cache:
        _same_device(self.pages, page_table, self.k_scale, self.v_scale)
        if page_table.dim() != 2 or page_table.shape[0] < B:
            raise SpecError("page_table must be [B, max_pages]")
        return _Cache(_dev(self.pages, "pages", torch.uint8), self.n_pages, self.page_tokens, self.H,
                      self.D, _dev(self.k_scale, "k_scale", torch.float32),
                      _dev(self.v_scale, "v_scale", torch.float32), int(B),
                      int(page_table.shape[1]), _dev(page_table, "page_table", torch.int32))


def new_cache(n_pages: int, H: int, D: int, page_tokens: int = 64, device=None, k_scale=None,
              v_scale=None) -> PagedCache:
    """An empty pool: n_pages pages of page_tokens tokens (a multiple of 32)
    for H kv heads of D channels."""
    if D not in HEAD_CHANNELS or page_tokens < BLOCK_TOKENS or page_tokens % BLOCK_TOKENS:
        raise SpecError("D must be one of %s and page_tokens a multiple of 32" % (HEAD_CHANNELS,))
    pages = torch.zeros(n_pages, H, page_tokens // BLOCK_TOKENS, 36 * D, dtype=torch.uint8,
                        device=device or "cuda")
    return PagedCache(pages, k_scale, v_scale)


class CacheCall:
    """A library call with its arguments marshalled: calling it launches on the
    current stream (or `stream`) and returns its results.  Keeps its tensors alive.

    Its results, and a workspace that it made itself, belong to the stream that it
    was prepared for.  The first call on another stream waits for that workspace's
    zeros, and from then on no memory of the call is given away before that stream is
    through with it.  (Inputs have to be ready on the stream of the call, as for any
    launch; a call that a graph captures is ordered by whoever replays it.)"""

    def __init__(self, fn, args, result, keep, device, known, ready):
        self._fn, self._args, self._result, self._keep = fn, args, result, keep
        self._device = device
        self._known, self._ready = known, ready      # streams that the tensors are safe on; the zeros' event

    def __call__(self, stream=None):
        s = torch.cuda.current_stream(self._device) if stream is None else stream
        if s.cuda_stream not in self._known:
            self._adopt(s)
        rc = self._fn(*self._args, s.cuda_stream)
        if rc:
            _check(rc)
        return self._result

    def _adopt(self, s):
        with torch.cuda.stream(s):
            if torch.cuda.is_current_stream_capturing():
                return
        if self._ready is not None:
            s.wait_event(self._ready)
        for t in _tensors((self._keep, self._result)):
            t.record_stream(s)
        self._known.add(s.cuda_stream)


def _run(fn, args, result, keep, device, prepared, stream, zeroed=False):
    """The call, or a handle of it where `prepared`.  Results (and `zeroed`: a
    workspace) were made under _on(stream), so that their memory is `stream`'s from
    the start."""
    here = torch.cuda.current_stream(device)
    away = stream is not None and stream.cuda_stream != here.cuda_stream
    ready = None
    if prepared and zeroed:
        with _on(stream):
            if not torch.cuda.is_current_stream_capturing():
                ready = torch.cuda.Event()
                ready.record()
    call = CacheCall(fn, args, result, keep, device, set() if away else {here.cuda_stream}, ready)
    if prepared:
        return call
    call(stream if away else here)
    if away:
        for t in _tensors(result):
            t.record_stream(here)        # the caller goes on with them here
    return result


def _same_device(a, *others):
    if not a.is_cuda:
        raise SpecError("the cache must be on a CUDA device")
    if a.device.index != torch.cuda.current_device():
        raise SpecError("the cache is on %s but the current device is cuda:%d"
                        % (a.device, torch.cuda.current_device()))
    for t in others:
        if t is not None and t.device != a.device:
            raise SpecError("tensors on different devices: %s and %s" % (a.device, t.device))


def _float_code(dtype) -> int:
    if dtype not in (torch.float32, torch.bfloat16):
        raise SpecError("rows must be float32 or bfloat16, got %s" % dtype)
    return SPEC_BF16 if dtype == torch.bfloat16 else SPEC_F32


def _heads(x: torch.Tensor, what: str, D: int):
    """Pointer and (row, head) strides of a [rows, heads, D] tensor."""
    if not x.is_cuda:
        raise SpecError("%s must be a CUDA tensor" % what)
    if x.dim() != 3 or x.shape[2] != D or x.stride(2) != 1:
        raise SpecError("%s must be [rows, heads, %d] with contiguous channels" % (what, D))
    return x.data_ptr(), x.stride(0), x.stride(1)


def _paged(x, what: str, cache: PagedCache, dtype):
    if x is not None and x.numel() != cache.n_pages * cache.page_tokens:
        raise SpecError("%s must be [n_pages, page_tokens]" % what)
    return _dev(x, what, dtype)


def _per_request(x, what: str, n: int, dtype=torch.int32):
    if x is not None and x.numel() < n:
        raise SpecError("%s needs %d entries" % (what, n))
    return _dev(x, what, dtype)


def cache_append(cache: PagedCache, k, v, cu_rows, start, page_table, *, B: int, max_rows: int,
                 score=None, slot_pos=None, pos0=None, status=None, prepared: bool = False,
                 stream=None):
    """spec_cache_append: quantise rows cu_rows[b] .. of k, v [R_cap, H, D] and
    write them to slots start[b] .. of request b; score (zeroed) and slot_pos
    (pos0[b] + i, default the slot) of those slots too when given.  max_rows
    bounds the rows of one request.  Returns the cache."""
    L = load_library()
    _same_device(cache.pages, k, v, cu_rows, start, score, slot_pos, pos0, status)
    if k.dtype != v.dtype or k.shape != v.shape or k.dim() != 3 or k.shape[1] != cache.H:
        raise SpecError("k and v must be [rows, %d, %d] of one dtype" % (cache.H, cache.D))
    view = cache._view(page_table, B)
    kp, kr, kh = _heads(k, "k", cache.D)
    vp, vr, vh = _heads(v, "v", cache.D)
    rows = _Rows(kp, vp, _float_code(k.dtype), kr, kh, vr, vh, k.shape[0], int(max_rows),
                 _per_request(cu_rows, "cu_rows", B + 1), _per_request(start, "start", B),
                 _paged(score, "score", cache, torch.float32),
                 _paged(slot_pos, "slot_pos", cache, torch.int32),
                 _per_request(pos0, "pos0", B), _dev(status, "status", torch.int32))
    keep = (cache, k, v, cu_rows, start, page_table, score, slot_pos, pos0, status, view, rows)
    return _run(L.spec_cache_append, (C.byref(view), C.byref(rows)), cache, keep, k.device, prepared, stream)


def cache_read(cache: PagedCache, cu_rows, start, page_table, *, B: int, max_rows: int,
               R_cap: Optional[int] = None, dtype=torch.float32, status=None,
               prepared: bool = False, stream=None):
    """spec_cache_read: the values of slots start[b] .. of every request, packed
    by cu_rows, as {"k", "v"} [R_cap, H, D].  Rows of no request are left
    unwritten."""
    L = load_library()
    _same_device(cache.pages, cu_rows, start, status)
    view = cache._view(page_table, B)
    R_cap = B * max_rows if R_cap is None else int(R_cap)
    shape = (R_cap, cache.H, cache.D)
    with _on(stream):
        res = {n: torch.empty(shape, dtype=dtype, device=cache.pages.device) for n in ("k", "v")}
    kp, kr, kh = _heads(res["k"], "k", cache.D)
    vp, vr, vh = _heads(res["v"], "v", cache.D)
    rows = _Rows(kp, vp, _float_code(dtype), kr, kh, vr, vh, R_cap, int(max_rows),
                 _per_request(cu_rows, "cu_rows", B + 1), _per_request(start, "start", B), None,
                 None, None, _dev(status, "status", torch.int32))
    keep = (cache, cu_rows, start, page_table, status, view, rows)
    return _run(L.spec_cache_read, (C.byref(view), C.byref(rows)), res, keep, cache.pages.device, prepared, stream)


def cache_workspace_bytes(B: int, k_max: int, Hq: int, H: int, D: int, max_len: int) -> int:
    return int(load_library().spec_cache_workspace_bytes(int(B), int(k_max), int(Hq), int(H), int(D),
                                                         int(max_len)))


def new_cache_workspace(cache: PagedCache, page_table, *, B: int, k_max: int, Hq: int,
                        max_len: Optional[int] = None) -> torch.Tensor:
    """Zero-filled workspace of cache_attend (reusable, stream-ordered)."""
    n = cache_workspace_bytes(B, k_max, Hq, cache.H, cache.D,
                              max_len or page_table.shape[1] * cache.page_tokens)
    if n == 0:
        raise SpecError("invalid cache workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=cache.pages.device)


def _attention(cache, q, cu_rows, cache_len, page_table, B, k_max, max_len, scale, cap, slopes,
               window, prefix, slot_pos, status, *more):
    _same_device(cache.pages, q, cu_rows, cache_len, slopes, slot_pos, status, *more)
    view = cache._view(page_table, B)
    qp, qr, qh = _heads(q, "q", cache.D)
    return view, _Attention(
        qp, _float_code(q.dtype), qr, qh, q.shape[1], q.shape[0], int(k_max),
        _per_request(cu_rows, "cu_rows", B + 1), _per_request(cache_len, "cache_len", B),
        int(max_len or 0), 1.0 / math.sqrt(cache.D) if scale is None else float(scale), float(cap),
        _per_request(slopes, "slopes", q.shape[1], torch.float32), int(window), int(prefix),
        _paged(slot_pos, "slot_pos", cache, torch.int32), _dev(status, "status", torch.int32))


def cache_attend(cache: PagedCache, q, cu_rows, cache_len, page_table, *, B: int, k_max: int,
                 max_len: Optional[int] = None, scale: Optional[float] = None, cap: float = 0.0,
                 slopes=None, window: int = 0, prefix: int = 0, slot_pos=None, workspace=None,
                 status=None, prepared: bool = False, stream=None):
    """spec_cache_attend: softmax attention of the packed rows q [R_cap, Hq, D]
    over each request's first cache_len[b] slots, causal among the rows (the
    last row sees every slot).  scale defaults to 1/sqrt(D); cap, slopes,
    window and prefix as in spec_cache.h.  Returns {"out" [R_cap, Hq, D],
    "lse" [R_cap, Hq]}; rows of no request are left unwritten."""
    L = load_library()
    view, attn = _attention(cache, q, cu_rows, cache_len, page_table, B, k_max, max_len, scale, cap,
                            slopes, window, prefix, slot_pos, status, workspace)
    with _on(stream):
        ws = workspace if workspace is not None else new_cache_workspace(
            cache, page_table, B=B, k_max=k_max, Hq=q.shape[1], max_len=max_len)
        res = {"out": torch.empty(q.shape, dtype=q.dtype, device=q.device),
               "lse": torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)}
    keep = (cache, q, cu_rows, cache_len, page_table, slopes, slot_pos, status, ws, view, attn)
    args = (C.byref(view), C.byref(attn), res["out"].data_ptr(), res["lse"].data_ptr(),
            _dev(ws, "workspace", torch.uint8), ws.numel())
    return _run(L.spec_cache_attend, args, res, keep, q.device, prepared, stream, zeroed=workspace is None)


def cache_weights(cache: PagedCache, q, lse, cu_rows, cache_len, page_table, score, *, B: int,
                  k_max: int, max_len: Optional[int] = None, scale: Optional[float] = None,
                  cap: float = 0.0, slopes=None, window: int = 0, prefix: int = 0, slot_pos=None,
                  status=None, prepared: bool = False, stream=None):
    """spec_cache_weights: add to score [n_pages, page_tokens] the attention
    weight that each slot got from the rows of q, whose lse cache_attend gave
    (same options); -inf there leaves a row out, as one of a rejected draft.  Returns
    score."""
    L = load_library()
    view, attn = _attention(cache, q, cu_rows, cache_len, page_table, B, k_max, max_len, scale, cap,
                            slopes, window, prefix, slot_pos, status, lse, score)
    if lse.numel() != q.shape[0] * q.shape[1]:
        raise SpecError("lse must be [rows, Hq]")
    keep = (cache, q, lse, cu_rows, cache_len, page_table, score, slopes, slot_pos, status, view, attn)
    args = (C.byref(view), C.byref(attn), _dev(lse, "lse", torch.float32),
            _paged(score, "score", cache, torch.float32))
    return _run(L.spec_cache_weights, args, score, keep, q.device, prepared, stream)


def cache_evict(cache: PagedCache, score, cache_len, page_table, dst_table, *, B: int, budget: int,
                recent: int = 0, slot_pos=None, status=None, prepared: bool = False, stream=None):
    """spec_cache_evict: keep the `recent` newest slots of each request and its
    highest scores up to `budget`, moved in order to the pages of dst_table
    (with score and slot_pos).  Returns {"kept" [B, budget], "new_len" [B]}."""
    L = load_library()
    _same_device(cache.pages, score, cache_len, dst_table, slot_pos, status)
    view = cache._view(page_table, B)
    if dst_table.dim() != 2 or dst_table.shape[0] < B:
        raise SpecError("dst_table must be [B, pages]")
    dev = cache.pages.device
    with _on(stream):
        res = {"kept": torch.empty(B, int(budget), dtype=torch.int32, device=dev),
               "new_len": torch.empty(B, dtype=torch.int32, device=dev)}
    ev = _Eviction(_paged(score, "score", cache, torch.float32),
                   _paged(slot_pos, "slot_pos", cache, torch.int32),
                   _per_request(cache_len, "cache_len", B), int(budget), int(recent),
                   _dev(dst_table, "dst_table", torch.int32), int(dst_table.shape[1]),
                   res["kept"].data_ptr(), res["new_len"].data_ptr(),
                   _dev(status, "status", torch.int32))
    keep = (cache, score, cache_len, page_table, dst_table, slot_pos, status, view, ev)
    return _run(L.spec_cache_evict, (C.byref(view), C.byref(ev)), res, keep, dev, prepared, stream)
