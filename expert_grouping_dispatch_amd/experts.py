"""Binding of the experts' products (``include/moe_experts.h``): dispatch and
rows in 8-bit integers, the grouped int8 product, the whole layer for a few
tokens.  Same manner as the package: checks, pointers, the current stream."""
from __future__ import annotations

import ctypes

import torch

from . import _check, _device_of, _i32, _i64, _id_dtype, _need, _p, _ptr, _rows_and_restore, _stream, _sz, _u32, lib

MATMUL_SWIGLU = 1          # flags bit of moe_expert_matmul_i8: gate and up rows, out = silu(gate) * up
MATMUL_MAX_DEPTH = 131056  # largest depth of moe_expert_matmul_i8
FEW_MAX_SLOTS = 2048       # largest n_rows * top_k of moe_layer_few

lib.moe_dispatch_i8.argtypes = [_p, _i64, _i32, _i32, _p, _p, _p, _i64, _p]
lib.moe_dispatch_i8.restype = ctypes.c_int
lib.moe_quantize_i8.argtypes = [_p, _i64, _i32, _p, _p, _p, _p]
lib.moe_quantize_i8.restype = ctypes.c_int
lib.moe_expert_matmul_i8.argtypes = [_p, _p, _i64, _p, _p, _i32, _p, _p, _i32, _i32, _u32, _p, _p]
lib.moe_expert_matmul_i8.restype = ctypes.c_int
lib.moe_layer_few_workspace_bytes.argtypes = [_i64, _i32, _i32]
lib.moe_layer_few_workspace_bytes.restype = _sz
for _f in (lib.moe_layer_few, lib.moe_layer_few_i64):
    _f.argtypes = [_p, _i64, _i32, _i32, _p, _p, _p, _i32, _i32, _p, _p, _p, _p, _i32, _p, _p, _sz, _p]
    _f.restype = ctypes.c_int


def alloc_quantized(n_rows: int, hidden: int, device):
    """(payload int8 [n_rows, hidden], scales fp32 [n_rows]) buffers for moe_dispatch_i8 and moe_quantize_i8."""
    return (torch.empty((n_rows, hidden), dtype=torch.int8, device=device),
            torch.empty(n_rows, dtype=torch.float32, device=device))


def _quantized(q, scales, hidden, dev, names):
    _need(q, names[0], torch.int8, dev)
    _need(scales, names[1], torch.float32, dev)
    if q.dim() != 2 or q.shape[1] != hidden or scales.numel() != q.shape[0]:
        raise ValueError(f"{names[0]} must be [rows, {hidden}] and {names[1]} [rows]")


def moe_dispatch_i8(input_tokens: torch.Tensor, top_k: int, restore_token_order: torch.Tensor, out_q: torch.Tensor,
                    out_scales: torch.Tensor) -> None:
    """Token rows as int8 with a scale each, at every position their slots map to."""
    dev = _device_of(input_tokens)
    n, h = _rows_and_restore(input_tokens, restore_token_order, top_k, dev)
    _quantized(out_q, out_scales, h, dev, ("out_q", "out_scales"))
    with torch.cuda.device(dev):
        _check(lib.moe_dispatch_i8(_ptr(input_tokens), n, h, int(top_k), _ptr(restore_token_order), _ptr(out_q),
                                   _ptr(out_scales), out_q.shape[0], _stream(dev)), "moe_dispatch_i8")


def moe_quantize_i8(x: torch.Tensor, out_q: torch.Tensor, out_scales: torch.Tensor,
                    row_count: torch.Tensor = None) -> None:
    """Rows of x (bf16 [rows, hidden]) as int8 with a scale each.  ``row_count`` (uint32 [1] on the device, for
    instance ``expert_start_indices[-1:]``) limits the rows without the host knowing."""
    dev = _device_of(x)
    _need(x, "x", torch.bfloat16, dev)
    if x.dim() != 2:
        raise ValueError("x must be [rows, hidden]")
    _quantized(out_q, out_scales, x.shape[1], dev, ("out_q", "out_scales"))
    if out_q.shape[0] != x.shape[0]:
        raise ValueError("out_q must have x's rows")
    count = ctypes.c_void_p(0)
    if row_count is not None:
        _need(row_count, "row_count", torch.uint32, dev)
        if row_count.numel() != 1:
            raise ValueError("row_count must have one element")
        count = _ptr(row_count)
    with torch.cuda.device(dev):
        _check(lib.moe_quantize_i8(_ptr(x), x.shape[0], x.shape[1], count, _ptr(out_q), _ptr(out_scales),
                                   _stream(dev)), "moe_quantize_i8")


def moe_expert_matmul_i8(a_q: torch.Tensor, a_scales: torch.Tensor, expert_start_indices: torch.Tensor,
                         expert_ids: torch.Tensor, w_q: torch.Tensor, w_scales: torch.Tensor, out: torch.Tensor,
                         flags: int = 0) -> None:
    """Every active expert's product over its rows of the expert-contiguous buffer; w_q is int8 [E, n, depth]
    (n = 2 * out.shape[1] with MATMUL_SWIGLU, gate rows first), w_scales fp32 [E, n]."""
    dev = _device_of(a_q)
    if a_q.dim() != 2:
        raise ValueError("a_q must be [rows, depth]")
    _quantized(a_q, a_scales, a_q.shape[1], dev, ("a_q", "a_scales"))
    _need(w_q, "w_q", torch.int8, dev)
    _need(w_scales, "w_scales", torch.float32, dev)
    _need(out, "out", torch.bfloat16, dev)
    _need(expert_start_indices, "expert_start_indices", torch.uint32, dev)
    _need(expert_ids, "expert_ids", torch.int32, dev)
    if w_q.dim() != 3 or w_q.shape[2] != a_q.shape[1] or tuple(w_scales.shape) != tuple(w_q.shape[:2]):
        raise ValueError("w_q must be [E, n, depth] and w_scales [E, n]")
    e, wide = w_q.shape[:2]
    n_out = wide // 2 if flags & MATMUL_SWIGLU else wide
    if (flags & MATMUL_SWIGLU) and wide % 2:
        raise ValueError("w_q must hold as many up rows as gate rows")
    if out.dim() != 2 or tuple(out.shape) != (a_q.shape[0], n_out):
        raise ValueError(f"out must be [{a_q.shape[0]}, {n_out}]")
    if expert_start_indices.numel() != e + 1 or expert_ids.numel() != e:
        raise ValueError("expert_start_indices must have E+1 elements and expert_ids E")
    with torch.cuda.device(dev):
        _check(lib.moe_expert_matmul_i8(_ptr(a_q), _ptr(a_scales), a_q.shape[0], _ptr(expert_start_indices),
                                        _ptr(expert_ids), e, _ptr(w_q), _ptr(w_scales), n_out, a_q.shape[1],
                                        int(flags), _ptr(out), _stream(dev)), "moe_expert_matmul_i8")


def moe_layer_few_workspace_bytes(n_rows: int, top_k: int, inter: int) -> int:
    return int(lib.moe_layer_few_workspace_bytes(int(n_rows), int(top_k), int(inter)))


def alloc_layer_few(n_rows: int, top_k: int, inter: int, device) -> torch.Tensor:
    """The workspace of moe_layer_few."""
    n = moe_layer_few_workspace_bytes(n_rows, top_k, inter)
    if n == 0:
        raise ValueError("n_rows / top_k / inter out of range")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_layer_few(x: torch.Tensor, topk_ids: torch.Tensor, router_weights: torch.Tensor, w_gate_up: torch.Tensor,
                  w_down: torch.Tensor, output_tokens: torch.Tensor, workspace: torch.Tensor,
                  gate_up_scales: torch.Tensor = None, down_scales: torch.Tensor = None,
                  real_token_count: torch.Tensor = None, tp_rank: int = 0) -> None:
    """The whole layer for up to FEW_MAX_SLOTS slots: bf16 weights, or int8 weights with a scale per output
    channel.  w_gate_up is [E, 2*inter, hidden] (gate rows first), w_down [E, hidden, inter]."""
    dev = _device_of(x)
    _need(x, "x", torch.bfloat16, dev)
    dt = _id_dtype(topk_ids, "topk_ids")
    _need(topk_ids, "topk_ids", dt, dev)
    _need(router_weights, "router_weights", torch.float32, dev)
    _need(output_tokens, "output_tokens", torch.bfloat16, dev)
    _need(workspace, "workspace", torch.uint8, dev)
    if x.dim() != 2 or topk_ids.dim() != 2 or topk_ids.shape[0] != x.shape[0]:
        raise ValueError("x must be [N, hidden] and topk_ids [N, top_k]")
    if tuple(router_weights.shape) != tuple(topk_ids.shape) or tuple(output_tokens.shape) != tuple(x.shape):
        raise ValueError("router_weights must be [N, top_k] and output_tokens [N, hidden]")
    n, h = x.shape
    if (gate_up_scales is None) != (down_scales is None):
        raise ValueError("gate_up_scales and down_scales come together")
    wdt = torch.bfloat16 if gate_up_scales is None else torch.int8
    _need(w_gate_up, "w_gate_up", wdt, dev)
    _need(w_down, "w_down", wdt, dev)
    if w_down.dim() != 3 or w_down.shape[1] != h:
        raise ValueError("w_down must be [E, hidden, inter]")
    e, _, inter = w_down.shape
    if tuple(w_gate_up.shape) != (e, 2 * inter, h):
        raise ValueError("w_gate_up must be [E, 2*inter, hidden]")
    sg = sd = cnt = ctypes.c_void_p(0)
    if gate_up_scales is not None:
        _need(gate_up_scales, "gate_up_scales", torch.float32, dev)
        _need(down_scales, "down_scales", torch.float32, dev)
        if tuple(gate_up_scales.shape) != (e, 2 * inter) or tuple(down_scales.shape) != (e, h):
            raise ValueError("gate_up_scales must be [E, 2*inter] and down_scales [E, hidden]")
        sg, sd = _ptr(gate_up_scales), _ptr(down_scales)
    if real_token_count is not None:
        _need(real_token_count, "real_token_count", torch.int32, dev)
        if real_token_count.numel() != 1:
            raise ValueError("real_token_count must have one element")
        cnt = _ptr(real_token_count)
    fn = lib.moe_layer_few if dt == torch.int32 else lib.moe_layer_few_i64
    with torch.cuda.device(dev):
        _check(fn(_ptr(x), n, h, topk_ids.shape[1], _ptr(topk_ids), _ptr(router_weights), cnt, int(tp_rank), e,
                  _ptr(w_gate_up), sg, _ptr(w_down), sd, inter, _ptr(output_tokens), _ptr(workspace),
                  workspace.numel(), _stream(dev)), "moe_layer_few")
