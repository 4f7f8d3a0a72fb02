"""Binding of the verification of trees of drafts (include/spec_tree.h): the acceptance
of a path, and the adjustment of the rows' logits.

Argument marshalling only, like cache.py, and with the same `prepared` and `stream`.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from .binding import SpecError, _dev, _logits_dtype, _on, load_library
from .cache import _per_request, _run, _same_device


class _Tree(C.Structure):
    _fields_ = [("B", C.c_int32), ("k_max", C.c_int32), ("R_cap", C.c_int32), ("cu_rows", C.c_void_p),
                ("row_token", C.c_void_p), ("node_token", C.c_void_p), ("parent", C.c_void_p),
                ("accepted_len", C.c_void_p), ("out_tokens", C.c_void_p), ("next_token", C.c_void_p),
                ("path_rows", C.c_void_p), ("status", C.c_void_p)]


class _Rules(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("dtype", C.c_int32), ("V", C.c_int32), ("ld", C.c_int64), ("B", C.c_int32),
                ("k_max", C.c_int32), ("R_cap", C.c_int32), ("cu_rows", C.c_void_p), ("history", C.c_void_p),
                ("history_ld", C.c_int64), ("history_cap", C.c_int32), ("n_tokens", C.c_void_p),
                ("n_prompt", C.c_void_p), ("repetition", C.c_void_p), ("frequency", C.c_void_p),
                ("presence", C.c_void_p), ("node_token", C.c_void_p), ("parent", C.c_void_p),
                ("bias_cu", C.c_void_p), ("bias_ids", C.c_void_p), ("bias_values", C.c_void_p),
                ("n_bias", C.c_int32), ("allowed", C.c_void_p), ("allowed_ld", C.c_int64),
                ("n_allowed", C.c_int32), ("allowed_row", C.c_void_p), ("status", C.c_void_p)]


def tree_accept(row_token, node_token, parent, cu_rows, *, B: int, k_max: int, status=None, prepared: bool = False,
                stream=None) -> dict:
    """spec_tree_accept: follow the target's tokens (row_token [R_cap]) from each request's
    root through its tree of drafts (node_token, parent [R_cap]).  Returns {"accepted_len" [B],
    "out_tokens" [B, k_max + 1], "next_token" [B], "path_rows" [B, k_max + 1]}: the packed rows of
    the root and the accepted nodes, the last one repeated."""
    L = load_library()
    _same_device(row_token, node_token, parent, cu_rows, status, what="row_token")
    R_cap, dev = row_token.numel(), row_token.device
    with _on(stream):
        res = {"accepted_len": torch.empty(B, dtype=torch.int32, device=dev),
               "out_tokens": torch.empty(B, k_max + 1, dtype=torch.int32, device=dev),
               "next_token": torch.empty(B, dtype=torch.int32, device=dev),
               "path_rows": torch.empty(B, k_max + 1, dtype=torch.int32, device=dev)}
    call = _Tree(int(B), int(k_max), R_cap, _per_request(cu_rows, "cu_rows", B + 1),
                 _dev(row_token, "row_token", torch.int32), _per_request(node_token, "node_token", R_cap),
                 _per_request(parent, "parent", R_cap), *[res[n].data_ptr() for n in res], _dev(status, "status", torch.int32))
    keep = (row_token, node_token, parent, cu_rows, status, call)
    return _run(L.spec_tree_accept, (C.byref(call),), res, keep, dev, prepared, stream)


def adjust_logits(logits, cu_rows, *, V: int, B: int, k_max: int, history=None, n_tokens=None, n_prompt=None,
                  repetition=None, frequency=None, presence=None, node_token=None, parent=None, bias_cu=None,
                  bias_ids=None, bias_values=None, allowed=None, allowed_row=None, out: Optional[torch.Tensor] = None,
                  status=None, prepared: bool = False, stream=None) -> dict:
    """spec_adjust_logits: penalties for the tokens of history [B, columns] (the first
    n_tokens[b], of them n_prompt[b] of the prompt) and of each row's path (node_token [R_cap], with
    parent a tree, else a chain), biases, and the masks allowed [n, ceil(V / 32)] (int32 words;
    allowed_row [R_cap]: the mask of each row, -1 for none) on logits [R_cap, >= V].  out: where
    the result goes (logits itself to adjust in place; a new tensor by default).  Returns
    {"logits": out}."""
    L = load_library()
    _same_device(logits, cu_rows, history, n_tokens, n_prompt, repetition, frequency, presence, node_token, parent,
                 bias_cu, bias_ids, bias_values, allowed, allowed_row, out, status, what="logits")
    code = _logits_dtype(logits)
    for x, what in [(logits, "logits"), (out, "out")]:
        if x is not None and (x.dim() != 2 or x.stride(1) != 1 or x.shape[1] < V):
            raise SpecError("%s must be 2-D [rows, >= V] with contiguous rows" % what)
    R_cap = logits.shape[0]
    if out is not None and (out.dtype != logits.dtype or out.shape[0] < R_cap):
        raise SpecError("out must have logits' dtype and rows")
    if history is not None and (history.dim() != 2 or history.shape[0] < B or history.dtype != torch.int32
                                or (history.shape[1] > 1 and history.stride(1) != 1)):
        raise SpecError("history must be int32 [B, tokens] with contiguous rows")
    if history is not None and n_tokens is None:
        raise SpecError("history needs n_tokens")
    if (bias_cu is None) != (bias_ids is None) or (bias_ids is None) != (bias_values is None):
        raise SpecError("bias_cu, bias_ids and bias_values go together")
    n_bias = 0 if bias_ids is None else bias_ids.numel()
    if n_bias and bias_values.numel() < n_bias:
        raise SpecError("bias_values needs %d entries" % n_bias)
    if allowed is not None and (allowed.dim() != 2 or allowed.stride(1) != 1 or allowed.dtype != torch.int32
                                or allowed.shape[1] < (V + 31) // 32 or allowed.shape[0] < 1):
        raise SpecError("allowed must be int32 [masks, ceil(V / 32)] with contiguous rows")
    f32 = lambda x, what: _per_request(x, what, B, torch.float32)
    with _on(stream):
        res = {"logits": out if out is not None else torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype,
                                                                         device=logits.device)}
    y = res["logits"]
    call = _Rules(logits.data_ptr(), code, int(V), logits.stride(0), int(B), int(k_max), R_cap,
                  _per_request(cu_rows, "cu_rows", B + 1), None if history is None else history.data_ptr(),
                  0 if history is None else history.stride(0), 0 if history is None else history.shape[1],
                  _per_request(n_tokens, "n_tokens", B), _per_request(n_prompt, "n_prompt", B),
                  f32(repetition, "repetition"), f32(frequency, "frequency"), f32(presence, "presence"),
                  _per_request(node_token, "node_token", R_cap), _per_request(parent, "parent", R_cap),
                  _per_request(bias_cu, "bias_cu", B + 1), _dev(bias_ids, "bias_ids", torch.int32),
                  _dev(bias_values, "bias_values", torch.float32), n_bias, None if allowed is None else allowed.data_ptr(),
                  0 if allowed is None else allowed.stride(0), 0 if allowed is None else allowed.shape[0],
                  _per_request(allowed_row, "allowed_row", R_cap), _dev(status, "status", torch.int32))
    keep = (logits, cu_rows, history, n_tokens, n_prompt, repetition, frequency, presence, node_token, parent, bias_cu,
            bias_ids, bias_values, allowed, allowed_row, out, status, call)
    return _run(L.spec_adjust_logits, (C.byref(call), y.data_ptr(), y.stride(0)), res, keep, logits.device, prepared, stream)
