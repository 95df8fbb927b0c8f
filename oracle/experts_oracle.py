"""Plain CPU oracle of the experts' products.  TEST INFRASTRUCTURE ONLY: it
shares no code with the HIP library.

  * quantize_i8 -- a = max(max |x|, 2^-118), scale = fl32(a/127),
    inv = fl32(127/a), q = fl32(x*inv) to the nearest integer, ties to even.
    Quotients and products are formed in 64 bits and rounded once: the product
    of a bf16 and an fp32 value is exact in 64 bits, and a 64-bit quotient of
    two fp32 values rounds to the fp32 quotient.  A row with an infinity or a
    NaN has scale NaN; its payload is unspecified, zeros here.
  * dispatch_i8 -- row p of the output is the quantised row of token
    token_expert_order[p] // top_k.
  * expert_values -- the fp32 values v of every row and weight row: the exact
    integer sum, rounded to fp32, times the row's scale, times the channel's,
    each product rounded once.
  * swiglu -- silu(gate) * up in 64 bits.
  * layer_few -- the whole layer in 64 bits, with a bound on how far a result
    formed as the kernels do may be from it (see there).
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import bf16_bits_to_f32

F32 = np.float32


def quantize_i8(x_bits: np.ndarray):
    x = bf16_bits_to_f32(x_bits).astype(np.float64)
    bad = ~np.isfinite(x).all(axis=1)
    x[bad] = 0.0
    a = np.maximum(np.abs(x).max(axis=1), 2.0 ** -118)
    scale = (a / 127.0).astype(F32)
    inv = (127.0 / a).astype(F32).astype(np.float64)
    q = np.rint((x * inv[:, None]).astype(F32).astype(np.float64))
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def dispatch_i8(x_bits: np.ndarray, token_expert_order: np.ndarray, top_k: int, n_routed: int):
    q, s = quantize_i8(x_bits)
    rows = token_expert_order[:n_routed].astype(np.int64) // top_k
    return q[rows], s[rows]


def expert_values(a_q: np.ndarray, a_scales: np.ndarray, w_q: np.ndarray, w_scales: np.ndarray) -> np.ndarray:
    """fp32 [rows, n] of one expert: a_q [rows, depth], w_q [n, depth]."""
    # integer sums below 2^53: exact in 64-bit floating point, whatever the order
    c = (a_q.astype(np.float64) @ w_q.astype(np.float64).T).astype(F32)
    return (c * a_scales[:, None].astype(F32)) * w_scales[None, :].astype(F32)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def swiglu(gate: np.ndarray, up: np.ndarray) -> np.ndarray:
    g, u = gate.astype(np.float64), up.astype(np.float64)
    return g * _sigmoid(g) * u


def layer_few(x: np.ndarray, ids: np.ndarray, router_weights: np.ndarray, w_gate_up: np.ndarray,
              w_down: np.ndarray):
    """(out, bound), both float64 [N, H], of weights and activations given as
    values.  ids outside [0, E) are unrouted.

    The bound counts, in units u = 2^-24 (half a step of fp32, relative):
      * a sum of n products in fp32, in any order: (n + 2) u times the sum of
        the magnitudes, two of them for a scale on the sum and the joining of
        parts;
      * silu's slope is below 1.1; its evaluation and the product with up:
        (|g| + 8) u relative (the exponent's argument, the exponential, a
        quotient and two products);
      * h as two bf16 values: half a step of what half a step left, 2^-16
        relative;
      * the output: 2^-8 relative;
      * the weighted sum: (top_k + 1) u.
    """
    u24, half = 2.0 ** -24, 2.0 ** -8
    n, hidden = x.shape
    inter = w_down.shape[2]
    x, rw = x.astype(np.float64), router_weights.astype(np.float64)
    out, bound, total = np.zeros((n, hidden)), np.zeros((n, hidden)), np.zeros((n, hidden))
    for t in range(n):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < w_gate_up.shape[0]:
                continue
            wgu, wd = w_gate_up[e].astype(np.float64), w_down[e].astype(np.float64)
            v, mag = wgu @ x[t], np.abs(wgu) @ np.abs(x[t])
            dv = (hidden + 2) * u24 * mag
            g, up, dg, du = v[:inter], v[inter:], dv[:inter], dv[inter:]
            h = swiglu(g, up)
            dh = 1.1 * dg * (np.abs(up) + du) + np.abs(g * _sigmoid(g)) * du
            dh = dh + (np.abs(h) + dh) * (half * half + (np.abs(g) + 8) * u24)
            y = wd @ h
            dy = np.abs(wd) @ dh + (inter + 2) * u24 * (np.abs(wd) @ (np.abs(h) + dh))
            out[t] += rw[t, j] * y
            bound[t] += np.abs(rw[t, j]) * dy
            total[t] += np.abs(rw[t, j]) * (np.abs(y) + dy)
    bound += (ids.shape[1] + 1) * u24 * total
    bound += half * (np.abs(out) + bound) + 2.0 ** -133
    return out, bound
