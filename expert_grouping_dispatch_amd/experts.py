"""Binding of the experts' products (``include/moe_experts.h``): dispatch and
rows in 8-bit integers, the grouped int8 product, the whole layer for a few
tokens.  Same manner as the package: checks, pointers, the current stream."""
from __future__ import annotations

import ctypes

import torch

from . import _fast
from . import _check, _device_of, _fit32, _i32, _i64, _id_dtype, _need, _p, _sz, _u32, lib

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
for _f in (lib.moe_layer_few, lib.moe_layer_few_i64, lib.moe_layer_few_f8, lib.moe_layer_few_f8_i64):
    _f.argtypes = [_p, _i64, _i32, _i32, _p, _p, _p, _i32, _i32, _p, _p, _p, _p, _i32, _p, _p, _sz, _p]
    _f.restype = ctypes.c_int


# The smallest of these calls take a few microseconds on the GPU, so the checks
# are kept to what they must read: a tensor's type, its device's number, its
# layout and its address, and the stream comes as a number, without an object
# for it (row quantisation of 64 x 256: 6.4 us against 7.5 us a call).  Whether
# numbers fit 32 bits is first asked of all of them together.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _index_of(t: torch.Tensor) -> int:
    """The number of t's HIP device."""
    return t.get_device() if isinstance(t, torch.Tensor) and t.is_cuda else _device_of(t).index


def _at(t: torch.Tensor, name: str, dtype: torch.dtype, dev: int) -> int:
    """The address of a contiguous tensor of this type on device number dev."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()):
        _need(t, name, dtype, torch.device("cuda", dev))
    return t.data_ptr()


def _call(fn, what: str, dev: int, *args) -> None:
    if torch.cuda.current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status, what)


def alloc_quantized(n_rows: int, hidden: int, device):
    """(payload int8 [n_rows, hidden], scales fp32 [n_rows]) buffers for moe_dispatch_i8 and moe_quantize_i8."""
    return (torch.empty((n_rows, hidden), dtype=torch.int8, device=device),
            torch.empty(n_rows, dtype=torch.float32, device=device))


def _quantized(q, scales, hidden, dev, names):
    at = _at(q, names[0], torch.int8, dev), _at(scales, names[1], torch.float32, dev)
    if q.dim() != 2 or q.shape[1] != hidden or scales.numel() != q.shape[0]:
        raise ValueError(f"{names[0]} must be [rows, {hidden}] and {names[1]} [rows]")
    return at


def moe_dispatch_i8(input_tokens: torch.Tensor, top_k: int, restore_token_order: torch.Tensor, out_q: torch.Tensor,
                    out_scales: torch.Tensor) -> None:
    """Token rows as int8 with a scale each, at every position their slots map to."""
    if int(top_k) >> 31:
        _fit32(top_k)
    dev = _index_of(input_tokens)
    x = _at(input_tokens, "input_tokens", torch.bfloat16, dev)
    restore = _at(restore_token_order, "restore_token_order", torch.uint32, dev)
    if input_tokens.dim() != 2:
        raise ValueError("input_tokens must be [N, hidden]")
    n, h = input_tokens.shape
    if h >> 31:
        _fit32(h)
    if restore_token_order.numel() != n * top_k:
        raise ValueError("restore_token_order must have N*top_k elements")
    q, scales = _quantized(out_q, out_scales, h, dev, ("out_q", "out_scales"))
    _call(lib.moe_dispatch_i8, "moe_dispatch_i8", dev, x, n, h, int(top_k), restore, q, scales, out_q.shape[0])


def moe_quantize_i8(x: torch.Tensor, out_q: torch.Tensor, out_scales: torch.Tensor,
                    row_count: torch.Tensor = None) -> None:
    """Rows of x (bf16 [rows, hidden]) as int8 with a scale each.  ``row_count`` (uint32 [1] on the device, for
    instance ``expert_start_indices[-1:]``) limits the rows without the host knowing."""
    dev = _index_of(x)
    src = _at(x, "x", torch.bfloat16, dev)
    if x.dim() != 2:
        raise ValueError("x must be [rows, hidden]")
    n, h = x.shape
    if h >> 31:
        _fit32(h)
    q, scales = _quantized(out_q, out_scales, h, dev, ("out_q", "out_scales"))
    if out_q.shape[0] != n:
        raise ValueError("out_q must have x's rows")
    count = 0
    if row_count is not None:
        count = _at(row_count, "row_count", torch.uint32, dev)
        if row_count.numel() != 1:
            raise ValueError("row_count must have one element")
    _call(lib.moe_quantize_i8, "moe_quantize_i8", dev, src, n, h, count, q, scales)


def moe_expert_matmul_i8(a_q: torch.Tensor, a_scales: torch.Tensor, expert_start_indices: torch.Tensor,
                         expert_ids: torch.Tensor, w_q: torch.Tensor, w_scales: torch.Tensor, out: torch.Tensor,
                         flags: int = 0) -> None:
    """Every active expert's product over its rows of the expert-contiguous buffer; w_q is int8 [E, n, depth]
    (n = 2 * out.shape[1] with MATMUL_SWIGLU, gate rows first), w_scales fp32 [E, n]."""
    if int(flags) >> 31:
        _fit32(flags)
    dev = _index_of(a_q)
    if a_q.dim() != 2:
        raise ValueError("a_q must be [rows, depth]")
    rows, depth = a_q.shape
    a, sa = _quantized(a_q, a_scales, depth, dev, ("a_q", "a_scales"))
    w, sw = _at(w_q, "w_q", torch.int8, dev), _at(w_scales, "w_scales", torch.float32, dev)
    o = _at(out, "out", torch.bfloat16, dev)
    starts = _at(expert_start_indices, "expert_start_indices", torch.uint32, dev)
    ids = _at(expert_ids, "expert_ids", torch.int32, dev)
    if w_q.dim() != 3 or w_q.shape[2] != depth or w_scales.shape != w_q.shape[:2]:
        raise ValueError("w_q must be [E, n, depth] and w_scales [E, n]")
    e, wide = w_q.shape[:2]
    if (e | wide | depth) >> 31:
        _fit32(e, wide, depth)
    n_out = wide // 2 if flags & MATMUL_SWIGLU else wide
    if (flags & MATMUL_SWIGLU) and wide % 2:
        raise ValueError("w_q must hold as many up rows as gate rows")
    if out.dim() != 2 or out.shape != (rows, n_out):
        raise ValueError(f"out must be [{rows}, {n_out}]")
    if expert_start_indices.numel() != e + 1 or expert_ids.numel() != e:
        raise ValueError("expert_start_indices must have E+1 elements and expert_ids E")
    _call(lib.moe_expert_matmul_i8, "moe_expert_matmul_i8", dev, a, sa, rows, starts, ids, e, w, sw, n_out, depth,
          int(flags), o)


def moe_layer_few_workspace_bytes(n_rows: int, top_k: int, inter: int) -> int:
    """The workspace's size in bytes, 0 if a size is out of range."""
    if (int(n_rows) | int(top_k) | int(inter)) >> 31:
        return 0
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
    """The whole layer for up to FEW_MAX_SLOTS slots: bf16 weights, int8 weights with a scale per output channel, or
    e4m3 weights (float8_e4m3fn) with a scale per block of 128 x 128: gate_up_scales [E, 2*ceil(inter/128),
    ceil(hidden/128)], gate blocks first, and down_scales [E, ceil(hidden/128), ceil(inter/128)].  w_gate_up is
    [E, 2*inter, hidden] (gate rows first), w_down [E, hidden, inter]."""
    if isinstance(w_gate_up, torch.Tensor) and w_gate_up.dtype is torch.float8_e4m3fn:
        status = _fast.layer_few_f8(x, topk_ids, router_weights, w_gate_up, w_down, output_tokens, workspace,
                                    gate_up_scales, down_scales, real_token_count, tp_rank)
        if status >= 0:
            return _check(status, "moe_layer_few")
    if int(tp_rank) >> 31:
        _fit32(tp_rank)
    dev = _index_of(x)
    src = _at(x, "x", torch.bfloat16, dev)
    dt = _id_dtype(topk_ids, "topk_ids")
    ids = _at(topk_ids, "topk_ids", dt, dev)
    rw = _at(router_weights, "router_weights", torch.float32, dev)
    out = _at(output_tokens, "output_tokens", torch.bfloat16, dev)
    space = _at(workspace, "workspace", torch.uint8, dev)
    if x.dim() != 2 or topk_ids.dim() != 2 or topk_ids.shape[0] != x.shape[0]:
        raise ValueError("x must be [N, hidden] and topk_ids [N, top_k]")
    if router_weights.shape != topk_ids.shape or output_tokens.shape != x.shape:
        raise ValueError("router_weights must be [N, top_k] and output_tokens [N, hidden]")
    n, h = x.shape
    if (gate_up_scales is None) != (down_scales is None):
        raise ValueError("gate_up_scales and down_scales come together")
    f8 = isinstance(w_gate_up, torch.Tensor) and w_gate_up.dtype is torch.float8_e4m3fn
    if f8 and gate_up_scales is None:
        raise ValueError("e4m3 weights need gate_up_scales and down_scales")
    wdt = torch.float8_e4m3fn if f8 else torch.bfloat16 if gate_up_scales is None else torch.int8
    w1, w2 = _at(w_gate_up, "w_gate_up", wdt, dev), _at(w_down, "w_down", wdt, dev)
    if w_down.dim() != 3 or w_down.shape[1] != h:
        raise ValueError("w_down must be [E, hidden, inter]")
    e, _, inter = w_down.shape
    if (h | topk_ids.shape[1] | e | inter) >> 31:
        _fit32(h, topk_ids.shape[1], e, inter)
    if w_gate_up.shape != (e, 2 * inter, h):
        raise ValueError("w_gate_up must be [E, 2*inter, hidden]")
    sg = sd = count = 0
    if gate_up_scales is not None:
        sg = _at(gate_up_scales, "gate_up_scales", torch.float32, dev)
        sd = _at(down_scales, "down_scales", torch.float32, dev)
        if f8:
            hb, ib = -(-h // 128), -(-inter // 128)
            if gate_up_scales.shape != (e, 2 * ib, hb) or down_scales.shape != (e, hb, ib):
                raise ValueError(f"gate_up_scales must be [E, {2 * ib}, {hb}] and down_scales [E, {hb}, {ib}]")
        elif gate_up_scales.shape != (e, 2 * inter) or down_scales.shape != (e, h):
            raise ValueError("gate_up_scales must be [E, 2*inter] and down_scales [E, hidden]")
    if real_token_count is not None:
        count = _at(real_token_count, "real_token_count", torch.int32, dev)
        if real_token_count.numel() != 1:
            raise ValueError("real_token_count must have one element")
    if f8:
        fn = lib.moe_layer_few_f8 if dt == torch.int32 else lib.moe_layer_few_f8_i64
    else:
        fn = lib.moe_layer_few if dt == torch.int32 else lib.moe_layer_few_i64
    _call(fn, "moe_layer_few", dev, src, n, h,
          topk_ids.shape[1], ids, rw, count, int(tp_rank), e, w1, sg, w2, sd, inter, out, space, workspace.numel())
