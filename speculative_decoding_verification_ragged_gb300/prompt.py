"""Binding of the attention of whole prompts (include/spec_prompt.h).

Argument marshalling only, like cache.py, and with the same `prepared` and `stream`.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional

import torch

from .binding import SpecError, _dev, _on, load_library
from .cache import HEAD_CHANNELS, _float_code, _heads, _per_request, _run, _same_device


class _Prompt(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("dtype", C.c_int32), ("D", C.c_int32),
                ("Hq", C.c_int32), ("H", C.c_int32), ("q_row", C.c_int64), ("q_head", C.c_int64),
                ("k_row", C.c_int64), ("k_head", C.c_int64), ("v_row", C.c_int64), ("v_head", C.c_int64),
                ("B", C.c_int32), ("R_cap", C.c_int32), ("K_cap", C.c_int32), ("cu_rows", C.c_void_p),
                ("cu_keys", C.c_void_p), ("scale", C.c_float), ("cap", C.c_float), ("slopes", C.c_void_p),
                ("window", C.c_int32), ("prefix", C.c_int32), ("status", C.c_void_p)]


def prompt_workspace_bytes(Hq: int, H: int, D: int, dtype=torch.bfloat16) -> int:
    return int(load_library().spec_prompt_workspace_bytes(int(Hq), int(H), int(D), _float_code(dtype)))


def new_prompt_workspace(Hq: int, H: int, D: int, dtype=torch.bfloat16, device=None) -> torch.Tensor:
    """Zero-filled workspace of prompt_attend (reusable, stream-ordered)."""
    n = prompt_workspace_bytes(Hq, H, D, dtype)
    if n == 0:
        raise SpecError("invalid prompt workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def prompt_attend(q, k, v, cu_rows, *, B: int, cu_keys=None, scale: Optional[float] = None, cap: float = 0.0,
                  slopes=None, window: int = 0, prefix: int = 0, workspace=None, status=None,
                  prepared: bool = False, stream=None):
    """spec_prompt_attend: causal softmax attention of the packed prompts q [R_cap, Hq, D]
    over their own keys and values k, v [K_cap, H, D].  With cu_keys a request has keys
    cu_keys[b] .., and its rows are the last of them.  scale defaults to 1/sqrt(D); cap,
    slopes, window and prefix as in spec_prompt.h.  workspace: new_prompt_workspace's, which a caller
    keeps (without one, up to 20 MB are zeroed with every call).  Returns {"out" [R_cap, Hq, D],
    "lse" [R_cap, Hq]}; rows of no request are left unwritten."""
    L = load_library()
    _same_device(q, k, v, cu_rows, cu_keys, slopes, workspace, status, what="q")
    if q.dim() != 3 or q.shape[2] not in HEAD_CHANNELS:
        raise SpecError("q must be [rows, heads, D], D one of %s" % (HEAD_CHANNELS,))
    if k.dtype != q.dtype or v.dtype != q.dtype or k.dim() != 3 or k.shape != v.shape:
        raise SpecError("k and v must be [keys, kv heads, D] of q's dtype")
    Hq, D, H = q.shape[1], q.shape[2], k.shape[1]
    qp, qr, qh = _heads(q, "q", D)
    kp, kr, kh = _heads(k, "k", D)
    vp, vr, vh = _heads(v, "v", D)
    call = _Prompt(qp, kp, vp, _float_code(q.dtype), D, Hq, H, qr, qh, kr, kh, vr, vh, int(B), q.shape[0], k.shape[0],
                   _per_request(cu_rows, "cu_rows", B + 1), _per_request(cu_keys, "cu_keys", B + 1),
                   1.0 / math.sqrt(D) if scale is None else float(scale), float(cap),
                   _per_request(slopes, "slopes", Hq, torch.float32), int(window), int(prefix),
                   _dev(status, "status", torch.int32))
    with _on(stream):
        ws = workspace if workspace is not None else new_prompt_workspace(Hq, H, D, q.dtype, q.device)
        res = {"out": torch.empty(q.shape, dtype=q.dtype, device=q.device),
               "lse": torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)}
    keep = (q, k, v, cu_rows, cu_keys, slopes, status, ws, call)
    args = (C.byref(call), res["out"].data_ptr(), res["lse"].data_ptr(), _dev(ws, "workspace", torch.uint8), ws.numel())
    return _run(L.spec_prompt_attend, args, res, keep, q.device, prepared, stream, zeroed=workspace is None)
