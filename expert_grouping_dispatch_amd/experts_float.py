"""Binding of the experts' products in floating point
(``include/moe_experts_float.h``): the grouped products in bf16 and in e4m3
with a scale for each block of 128, dispatch and rows in e4m3.  Same manner as
``experts``; a call whose tensors are all as they should be goes to the library
from ``_fast`` (``csrc/binding.cpp``), which returns its status, or -1 for any
other call, whose arguments are then checked here one by one."""
from __future__ import annotations

import ctypes

import torch

from . import _check, _fit32, _i32, _i64, _p, _u32, lib
from . import _fast
from .experts import MATMUL_SWIGLU, _at, _call, _index_of

F8_BLOCK = 128  # values of a row, and weight rows, that share a scale
F8 = torch.float8_e4m3fn

lib.moe_expert_matmul.argtypes = [_p, _i64, _p, _p, _i32, _p, _i32, _i32, _u32, _p, _p]
lib.moe_expert_matmul.restype = ctypes.c_int
lib.moe_dispatch_f8.argtypes = [_p, _i64, _i32, _i32, _p, _p, _p, _i64, _p]
lib.moe_dispatch_f8.restype = ctypes.c_int
lib.moe_quantize_f8.argtypes = [_p, _i64, _i32, _p, _p, _p, _p]
lib.moe_quantize_f8.restype = ctypes.c_int
lib.moe_expert_matmul_f8.argtypes = [_p, _p, _i64, _p, _p, _i32, _p, _p, _i32, _i32, _u32, _p, _p]
lib.moe_expert_matmul_f8.restype = ctypes.c_int


def _blocks(n: int) -> int:
    return -(-n // F8_BLOCK)


def alloc_quantized_f8(n_rows: int, hidden: int, device):
    """(payload e4m3 [n_rows, hidden], scales fp32 [n_rows, ceil(hidden/128)]) buffers for moe_dispatch_f8 and
    moe_quantize_f8."""
    return (torch.empty((n_rows, hidden), dtype=F8, device=device),
            torch.empty((n_rows, _blocks(hidden)), dtype=torch.float32, device=device))


def _quantized(q, scales, hidden, dev, names):
    at = _at(q, names[0], F8, dev), _at(scales, names[1], torch.float32, dev)
    if q.dim() != 2 or q.shape[1] != hidden or scales.shape != (q.shape[0], _blocks(hidden)):
        raise ValueError(f"{names[0]} must be [rows, {hidden}] and {names[1]} [rows, {_blocks(hidden)}]")
    return at


def moe_dispatch_f8(input_tokens: torch.Tensor, top_k: int, restore_token_order: torch.Tensor, out_q: torch.Tensor,
                    out_scales: torch.Tensor) -> None:
    """Token rows as e4m3 with a scale for each 128 values, at every position their slots map to."""
    status = _fast.dispatch_f8(input_tokens, top_k, restore_token_order, out_q, out_scales)
    if status >= 0:
        return _check(status, "moe_dispatch_f8")
    _fit32(top_k)
    dev = _index_of(input_tokens)
    x = _at(input_tokens, "input_tokens", torch.bfloat16, dev)
    restore = _at(restore_token_order, "restore_token_order", torch.uint32, dev)
    if input_tokens.dim() != 2:
        raise ValueError("input_tokens must be [N, hidden]")
    n, h = input_tokens.shape
    _fit32(h)
    if restore_token_order.numel() != n * top_k:
        raise ValueError("restore_token_order must have N*top_k elements")
    q, scales = _quantized(out_q, out_scales, h, dev, ("out_q", "out_scales"))
    _call(lib.moe_dispatch_f8, "moe_dispatch_f8", dev, x, n, h, int(top_k), restore, q, scales, out_q.shape[0])


def moe_quantize_f8(x: torch.Tensor, out_q: torch.Tensor, out_scales: torch.Tensor,
                    row_count: torch.Tensor = None) -> None:
    """Rows of x (bf16 [rows, hidden]) as e4m3 with a scale for each 128 values.  ``row_count`` (uint32 [1] on the
    device, for instance ``expert_start_indices[-1:]``) limits the rows without the host knowing."""
    status = _fast.quantize_f8(x, out_q, out_scales, row_count)
    if status >= 0:
        return _check(status, "moe_quantize_f8")
    dev = _index_of(x)
    src = _at(x, "x", torch.bfloat16, dev)
    if x.dim() != 2:
        raise ValueError("x must be [rows, hidden]")
    n, h = x.shape
    _fit32(h)
    q, scales = _quantized(out_q, out_scales, h, dev, ("out_q", "out_scales"))
    if out_q.shape[0] != n:
        raise ValueError("out_q must have x's rows")
    count = 0
    if row_count is not None:
        count = _at(row_count, "row_count", torch.uint32, dev)
        if row_count.numel() != 1:
            raise ValueError("row_count must have one element")
    _call(lib.moe_quantize_f8, "moe_quantize_f8", dev, src, n, h, count, q, scales)


def _grouped(a, w, expert_start_indices, expert_ids, out, flags, dtype, dev, names):
    """What both grouped products check: the addresses of a, w, the groups and out, and the sizes."""
    pa = _at(a, names[0], dtype, dev)
    pw, o = _at(w, names[1], dtype, dev), _at(out, "out", torch.bfloat16, dev)
    starts = _at(expert_start_indices, "expert_start_indices", torch.uint32, dev)
    ids = _at(expert_ids, "expert_ids", torch.int32, dev)
    if a.dim() != 2:
        raise ValueError(f"{names[0]} must be [rows, depth]")
    rows, depth = a.shape
    if w.dim() != 3 or w.shape[2] != depth:
        raise ValueError(f"{names[1]} must be [E, n, depth]")
    e, n_out = w.shape[:2]
    _fit32(e, n_out, depth)
    if flags & MATMUL_SWIGLU:
        if n_out % 2:
            raise ValueError(f"{names[1]} must hold as many up rows as gate rows")
        n_out //= 2
    if out.dim() != 2 or out.shape != (rows, n_out):
        raise ValueError(f"out must be [{rows}, {n_out}]")
    if expert_start_indices.numel() != e + 1 or expert_ids.numel() != e:
        raise ValueError("expert_start_indices must have E+1 elements and expert_ids E")
    return pa, pw, starts, ids, o, rows, depth, e, n_out


def moe_expert_matmul(a: torch.Tensor, expert_start_indices: torch.Tensor, expert_ids: torch.Tensor, w: torch.Tensor,
                      out: torch.Tensor, flags: int = 0) -> None:
    """Every active expert's product over its rows of the expert-contiguous buffer, in bf16; w is [E, n, depth]
    (n = 2 * out.shape[1] with MATMUL_SWIGLU, gate rows first)."""
    status = _fast.expert_matmul(a, expert_start_indices, expert_ids, w, out, flags)
    if status >= 0:
        return _check(status, "moe_expert_matmul")
    _fit32(flags)
    dev = _index_of(a)
    pa, pw, starts, ids, o, rows, depth, e, n_out = _grouped(a, w, expert_start_indices, expert_ids, out, flags,
                                                             torch.bfloat16, dev, ("a", "w"))
    _call(lib.moe_expert_matmul, "moe_expert_matmul", dev, pa, rows, starts, ids, e, pw, n_out, depth, int(flags), o)


def moe_expert_matmul_f8(a_q: torch.Tensor, a_scales: torch.Tensor, expert_start_indices: torch.Tensor,
                         expert_ids: torch.Tensor, w_q: torch.Tensor, w_scales: torch.Tensor, out: torch.Tensor,
                         flags: int = 0) -> None:
    """The same in e4m3: a_scales is fp32 [rows, ceil(depth/128)], w_scales fp32 [E, ceil(n/128), ceil(depth/128)],
    with MATMUL_SWIGLU [E, 2 * ceil(out.shape[1]/128), ceil(depth/128)], the gate rows' blocks first."""
    status = _fast.expert_matmul_f8(a_q, a_scales, expert_start_indices, expert_ids, w_q, w_scales, out, flags)
    if status >= 0:
        return _check(status, "moe_expert_matmul_f8")
    _fit32(flags)
    dev = _index_of(a_q)
    pa, pw, starts, ids, o, rows, depth, e, n_out = _grouped(a_q, w_q, expert_start_indices, expert_ids, out, flags,
                                                             F8, dev, ("a_q", "w_q"))
    _, sa = _quantized(a_q, a_scales, depth, dev, ("a_q", "a_scales"))
    sw = _at(w_scales, "w_scales", torch.float32, dev)
    halves = 2 if flags & MATMUL_SWIGLU else 1
    if w_scales.shape != (e, halves * _blocks(n_out), _blocks(depth)):
        raise ValueError(f"w_scales must be [{e}, {halves * _blocks(n_out)}, {_blocks(depth)}]")
    _call(lib.moe_expert_matmul_f8, "moe_expert_matmul_f8", dev, pa, sa, rows, starts, ids, e, pw, sw, n_out, depth,
          int(flags), o)
