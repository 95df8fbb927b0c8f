"""What is measured of the experts' products in floating point: dispatch and rows in e4m3 with a scale for each
128 values, the grouped products in bf16 and in e4m3 with a scale for each block of 128, and the whole layer for a
few tokens with such weights.

``run`` computes a case in plain torch operations in 32 bits where ``own`` is
false, and through the framework's entry points where it is true.  ``exact``
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
BLOCK = 128


# ---- cases ------------------------------------------------------------------------------------------------


def listed():
    return [
        # dispatch: the tiny workload, where only latency counts, and a skewed prefill
        dict(name="dispatch tiny", op="dispatch", rows=64, real=64, hidden=256, experts=8, top_k=2, routing="uniform"),
        dict(name="dispatch prefill", op="dispatch", rows=4096, real=4096, hidden=7168, experts=256, top_k=8,
             routing="zipf"),
        # activations between the two products: a decode batch in its padded buffer, a long prefill with wide experts
        dict(name="quantize decode", op="quantize", rows=2048, real=776, hidden=2048),
        dict(name="quantize prefill", op="quantize", rows=16384, real=14000, hidden=14336),
        # bf16 products: a small odd batch over small experts, a prefill over few and wide ones (with its SwiGLU), the
        # second product of a skewed prefill, whose groups are ragged
        dict(name="bf16 odd", op="matmul", type="bf16", rows=24, real=13, experts=24, top_k=4, routing="uniform",
             depth=1040, out=528, swiglu=False),
        dict(name="bf16 prefill swiglu", op="matmul", type="bf16", rows=8192, real=7000, experts=8, top_k=2,
             routing="uniform", depth=4096, out=14336, swiglu=True),
        dict(name="bf16 prefill down", op="matmul", type="bf16", rows=4096, real=4096, experts=256, top_k=8,
             routing="zipf", depth=2048, out=7168, swiglu=False),
        # e4m3 products: a decode batch spread over many experts, the wide prefill, the second product of the largest
        # batch
        dict(name="f8 decode swiglu", op="matmul", type="f8", rows=256, real=97, experts=256, top_k=8,
             routing="uniform", depth=7168, out=2048, swiglu=True),
        dict(name="f8 prefill swiglu", op="matmul", type="f8", rows=8192, real=7000, experts=8, top_k=2,
             routing="uniform", depth=4096, out=14336, swiglu=True),
        dict(name="f8 stress down", op="matmul", type="f8", rows=65536, real=61440, experts=256, top_k=8,
             routing="hotcold", depth=2048, out=7168, swiglu=False),
        # whole layer: one token, a captured decode batch with padding rows
        dict(name="layer one token", op="layer", rows=1, real=1, hidden=4096, inter=14336, experts=8, top_k=2,
             routing="uniform"),
        dict(name="layer decode", op="layer", rows=256, real=97, hidden=7168, inter=2048, experts=256, top_k=8,
             routing="uniform"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    """A row length: a multiple of 16, spread over the logarithm; the last block of 128 is mostly a part of one."""
    return 16 * max(1, _spread(rng, lo, hi) // 16)


def draw(rng):
    while True:
        op = rng.choice(("dispatch", "quantize", "matmul", "matmul", "matmul", "layer", "layer"))
        if op == "quantize":
            rows = _spread(rng, 1, 32768)
            c = dict(op=op, rows=rows, real=rng.randint(0, rows), hidden=_wide(rng, 64, 16384))
            if c["rows"] * c["hidden"] <= 16384 * 14336:
                return c
            continue
        experts = _spread(rng, 4, 256)
        c = dict(op=op, rows=_spread(rng, 1, 256 if op == "layer" else 16384), experts=experts,
                 top_k=rng.randint(1, min(8, experts)), routing=rng.choice(("uniform", "zipf")))
        c["real"] = c["rows"] if rng.random() < 0.5 else rng.randint(1, c["rows"])
        slots = c["real"] * c["top_k"]
        if op == "dispatch":
            c["hidden"] = _wide(rng, 64, 8192)
            if c["rows"] * c["hidden"] <= 4096 * 7168:
                return c
        elif op == "matmul":
            c.update(type=rng.choice(("bf16", "f8")), depth=_wide(rng, 64, 8192), out=_wide(rng, 64, 8192),
                     swiglu=rng.random() < 0.5)
            wide = c["out"] * (2 if c["swiglu"] else 1)
            if experts * c["depth"] * wide <= 3.7e9 and slots * c["depth"] * wide <= 1e12:
                return c
        else:
            c.update(hidden=_wide(rng, 256, 8192), inter=_wide(rng, 128, 8192))
            if experts * c["hidden"] * c["inter"] <= 1.25e9:
                return c


def _blocks(n):
    return -(-n // BLOCK)


def _active(c):
    """How many experts get a row, on average over the draws of the routing."""
    if c["routing"] == "hotcold":
        return c["experts"] - 3
    if c["routing"] == "uniform":
        return c["experts"] * (1 - (1 - c["top_k"] / c["experts"]) ** c["real"])
    p = [(r + 1) ** -1.2 for r in range(c["experts"])]
    s = sum(p)
    return sum(1 - (1 - min(1.0, c["top_k"] * v / s)) ** c["real"] for v in p)


def work(case):
    c = case
    if c["op"] == "quantize":
        return {"bytes": c["real"] * (3 * c["hidden"] + 4 * _blocks(c["hidden"])) or 4,
                "flops": 3 * c["real"] * c["hidden"]}
    slots = c["real"] * c["top_k"]
    if c["op"] == "dispatch":
        return {"bytes": 2 * c["real"] * c["hidden"] + slots * (c["hidden"] + 4 * _blocks(c["hidden"])) +
                4 * c["rows"] * c["top_k"], "flops": 3 * c["real"] * c["hidden"]}
    if c["op"] == "matmul":
        halves = 2 if c["swiglu"] else 1
        wide = c["out"] * halves
        if c["type"] == "bf16":
            moved = 2 * slots * (c["depth"] + c["out"]) + _active(c) * wide * c["depth"] * 2
        else:
            moved = slots * (c["depth"] + 4 * _blocks(c["depth"]) + 2 * c["out"]) + _active(c) * (
                wide * c["depth"] + 4 * halves * _blocks(c["out"]) * _blocks(c["depth"]))
        return {"bytes": moved, "flops": 2 * slots * c["depth"] * wide}
    each = 3 * c["hidden"] * c["inter"] + 12 * _blocks(c["hidden"]) * _blocks(c["inter"])
    return {"bytes": _active(c) * each + 2 * (c["real"] + c["rows"]) * c["hidden"] + 8 * c["rows"] * c["top_k"],
            "flops": 6 * slots * c["hidden"] * c["inter"]}


# ---- inputs -----------------------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    """Normal values in `dtype`, drawn in pieces; e4m3 is what a block's scale leaves of them: its largest value at
    448, some four standard deviations in a block of 128 x 128 and under three in 128 values of a row."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat, step = out.view(-1), 1 << 27
    for at in range(0, flat.numel(), step):
        v = torch.randn(min(step, flat.numel() - at), generator=g, device=DEV).mul_(scale)
        flat[at:at + step] = v.clamp_(-448, 448).to(F8) if dtype == F8 else v
    return out


def _routing(c, g):
    """Distinct experts per token, as the router's top k gives them; padding rows are -1."""
    n, e, k = c["real"], c["experts"], c["top_k"]
    keys = -torch.log(-torch.log(torch.rand((n, e), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)))
    perm = torch.randperm(e, generator=g, device=DEV)
    if c["routing"] == "zipf":
        keys -= 1.2 * torch.log(torch.arange(1, e + 1, device=DEV).float())
    if c["routing"] == "hotcold":  # half of the slots on 26 experts, half on the others, three never chosen
        hot, rest = keys[:, :26].topk(k // 2)[1], keys[:, 26:e - 3].topk(k - k // 2)[1] + 26
        top = torch.cat((hot, rest), 1)
    else:
        top = keys.topk(k)[1]
    ids = torch.full((c["rows"], k), -1, dtype=torch.int32, device=DEV)
    ids[:n] = perm[top].int()
    return ids


def _indices(c, ids):
    """What moe_create_indices writes: slots in stable expert order, their inverse, starts of the active experts."""
    flat = ids.view(-1)
    routed = flat >= 0
    v = int(routed.sum())
    key = torch.where(routed, flat, torch.full_like(flat, c["experts"]))
    order = torch.sort(key, stable=True)[1]
    restore = torch.full((flat.numel(),), 0xFFFFFFFF, dtype=torch.int64, device=DEV)
    restore[order[:v]] = torch.arange(v, device=DEV)
    counts = torch.bincount(key.long(), minlength=c["experts"] + 1)[:c["experts"]]
    active = counts.nonzero().view(-1)
    starts = torch.full((c["experts"] + 1,), v, dtype=torch.int64, device=DEV)
    starts[0] = 0
    starts[1:active.numel() + 1] = counts[active].cumsum(0)
    expert_ids = torch.full((c["experts"],), -1, dtype=torch.int32, device=DEV)
    expert_ids[:active.numel()] = active.int()
    at = starts[:active.numel() + 1].tolist()
    groups = list(zip(active.tolist(), at, at[1:]))
    return dict(order=order, restore=restore.to(torch.uint32), starts=starts.to(torch.uint32), expert_ids=expert_ids,
                groups=groups, routed=v)


def _scales(g, shape, mean):
    return (0.5 + torch.rand(shape, generator=g, device=DEV)).mul_(mean)


W_SIGMA, A_SIGMA = 105.0, 165.0  # standard deviations of what the scales of weights and of activations leave


def _weights(g, experts, halves, n, depth):
    """e4m3 [experts, halves * n, depth] and their scales; each half has block rows of its own."""
    return (_normal(g, (experts, halves * n, depth), F8, W_SIGMA),
            _scales(g, (experts, halves * _blocks(n), _blocks(depth)), 1 / (W_SIGMA * depth ** 0.5)))


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=dict(case))
    if c["op"] == "quantize":
        s["x"] = _normal(g, (c["rows"], c["hidden"]), torch.bfloat16)
        s["count"] = torch.tensor([c["real"]], dtype=torch.int64, device=DEV).to(torch.uint32)
        s["out_q"] = torch.zeros((c["rows"], c["hidden"]), device=DEV).to(F8)
        s["out_scales"] = torch.zeros((c["rows"], _blocks(c["hidden"])), device=DEV)
        return s
    ids = _routing(c, g)
    slots = ids.numel()
    s.update(_indices(c, ids))
    if c["op"] == "dispatch":
        s["x"] = _normal(g, (c["rows"], c["hidden"]), torch.bfloat16)
        s["out_q"] = torch.zeros((slots, c["hidden"]), device=DEV).to(F8)
        s["out_scales"] = torch.zeros((slots, _blocks(c["hidden"])), device=DEV)
    elif c["op"] == "matmul":
        halves, depth = 2 if c["swiglu"] else 1, c["depth"]
        if c["type"] == "bf16":
            s["a"] = _normal(g, (slots, depth), torch.bfloat16)
            s["w"] = _normal(g, (c["experts"], halves * c["out"], depth), torch.bfloat16, depth ** -0.5)
        else:
            s["a"] = _normal(g, (slots, depth), F8, A_SIGMA)
            s["a_scales"] = _scales(g, (slots, _blocks(depth)), 1 / A_SIGMA)
            s["w"], s["w_scales"] = _weights(g, c["experts"], halves, c["out"], depth)
        s["out"] = torch.zeros((slots, c["out"]), dtype=torch.bfloat16, device=DEV)
    else:
        h, i, e = c["hidden"], c["inter"], c["experts"]
        s["ids"] = ids
        s["x"] = _normal(g, (c["rows"], h), torch.bfloat16)
        s["router_weights"] = torch.softmax(torch.randn(ids.shape, generator=g, device=DEV), 1)
        s["w_gate_up"], s["gate_up_scales"] = _weights(g, e, 2, i, h)
        s["w_down"], s["down_scales"] = _weights(g, e, 1, h, i)
        s["out"] = torch.zeros((c["rows"], h), dtype=torch.bfloat16, device=DEV)
        # four bytes for each slot and intermediate channel are enough for any size
        s["workspace"] = torch.empty(4 * slots * i + 256, dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ---------------------------------------------------------------------------------------------


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _calls(s, op)
    if op == "quantize":
        n = s["case"]["real"]
        q, scales = torch.zeros_like(s["out_q"]), torch.zeros_like(s["out_scales"])
        q[:n], scales[:n] = _quantized(s["x"][:n])
        return q, scales
    if op == "dispatch":
        q, scales = torch.zeros_like(s["out_q"]), torch.zeros_like(s["out_scales"])
        rows = s["order"][:s["routed"]] // s["case"]["top_k"]
        tq, ts = _quantized(s["x"])
        q[:s["routed"]], scales[:s["routed"]] = tq[rows], ts[rows]
        return q, scales
    if op == "matmul":
        return _products(s)
    return _layer(s)


def _calls(s, op):
    import expert_grouping_dispatch_amd as moe

    if op == "quantize":
        moe.moe_quantize_f8(s["x"], s["out_q"], s["out_scales"], row_count=s["count"])
        return s["out_q"], s["out_scales"]
    if op == "dispatch":
        moe.moe_dispatch_f8(s["x"], s["case"]["top_k"], s["restore"], s["out_q"], s["out_scales"])
        return s["out_q"], s["out_scales"]
    if op == "matmul":
        flags = moe.MATMUL_SWIGLU if s["case"]["swiglu"] else 0
        if s["case"]["type"] == "bf16":
            moe.moe_expert_matmul(s["a"], s["starts"], s["expert_ids"], s["w"], s["out"], flags=flags)
        else:
            moe.moe_expert_matmul_f8(s["a"], s["a_scales"], s["starts"], s["expert_ids"], s["w"], s["w_scales"],
                                     s["out"], flags=flags)
        return s["out"]
    moe.moe_layer_few(s["x"], s["ids"], s["router_weights"], s["w_gate_up"], s["w_down"], s["out"], s["workspace"],
                      gate_up_scales=s["gate_up_scales"], down_scales=s["down_scales"])
    return s["out"]


def _quantized(x):
    """Rows to e4m3 with a scale for each 128 values: the divisions in 64 bits and rounded once, the product with the
    inverse rounded to 32 bits before it is rounded to e4m3, as the format is defined."""
    rows, n = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -n % BLOCK)).view(rows, -1, BLOCK)
    largest = v.abs().amax(2).clamp(min=2.0 ** -116).double()
    q = (v * (448.0 / largest).float()[:, :, None]).to(F8)
    return q.view(rows, -1)[:, :n], (largest / 448.0).float()


def _silu_times(gate, up):
    return gate / (1 + torch.exp(-gate)) * up


def _values(q, scales, halves=1):
    """What e4m3 weights [halves * n, depth] stand for, a scale for each block of 128 x 128 of a half."""
    n, depth = q.shape[0] // halves, q.shape[1]
    per = scales.view(halves, _blocks(n), -1).repeat_interleave(BLOCK, 1)[:, :n].reshape(halves * n, -1)
    return q.float() * per.repeat_interleave(BLOCK, 1)[:, :depth]


def _products(s):
    c = s["case"]
    n, halves, depth = c["out"], 2 if c["swiglu"] else 1, c["depth"]
    out = torch.zeros_like(s["out"])
    for e, lo, hi in s["groups"]:
        a = s["a"][lo:hi].float()
        if c["type"] == "bf16":
            w = s["w"][e].float()
        else:
            a = a * s["a_scales"][lo:hi].repeat_interleave(BLOCK, 1)[:, :depth]
            w = _values(s["w"][e], s["w_scales"][e], halves)
        y = a @ w.t()
        out[lo:hi] = _silu_times(y[:, :n], y[:, n:]) if c["swiglu"] else y
    return out


def _layer(s):
    c = s["case"]
    k, i = c["top_k"], c["inter"]
    y = torch.zeros((c["rows"] * k, c["hidden"]), device=DEV)
    for e, lo, hi in s["groups"]:
        slots = s["order"][lo:hi]
        t = s["x"][slots // k].float() @ _values(s["w_gate_up"][e], s["gate_up_scales"][e], 2).t()
        y[slots] = _silu_times(t[:, :i], t[:, i:]) @ _values(s["w_down"][e], s["down_scales"][e]).t()
    return (y.view(c["rows"], k, -1) * s["router_weights"][:, :, None]).sum(1).to(torch.bfloat16)


# ---- from the definitions, in 64 bits -----------------------------------------------------------------------


def _e4m3(t):
    """The value of e4m3 next to t, |t| <= 448, in 64 bits: a step is 2^(exponent - 3), at least 2^-9; ties go to the
    even multiple."""
    exponent = torch.frexp(t)[1].clamp(min=-5) - 1
    step = torch.exp2(exponent.double() - 3)
    low = torch.floor(t / step)
    above = t / step - low
    return (low + ((above > 0.5) | ((above == 0.5) & (low % 2 != 0))).double()) * step


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("quantize", "dispatch"):
        # a = max(|x|, 2^-116) over a block, scale = fl32(a / 448), q = e4m3(fl32(x * fl32(448 / a)))
        x = s["x"].double()
        q = torch.zeros_like(x)
        scales = torch.zeros((x.shape[0], _blocks(x.shape[1])), dtype=torch.float64, device=DEV)
        for b in range(scales.shape[1]):
            v = x[:, b * BLOCK:(b + 1) * BLOCK]
            a = torch.maximum(v.max(1)[0], -v.min(1)[0]).clamp(min=2.0 ** -116)
            inverse = (448 / a).float().double()
            q[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3((v * inverse.unsqueeze(1)).float().double())
            scales[:, b] = (a / 448).float().double()
        if c["op"] == "quantize":
            beyond = torch.arange(c["rows"], device=DEV) >= c["real"]
            q[beyond], scales[beyond] = 0, 0
            return q, scales
        at = s["restore"].to(torch.int64)
        slot = (at != 0xFFFFFFFF).nonzero().view(-1)
        out_q = torch.zeros(s["out_q"].shape, dtype=torch.float64, device=DEV)
        out_scales = torch.zeros(s["out_scales"].shape, dtype=torch.float64, device=DEV)
        token = torch.div(slot, c["top_k"], rounding_mode="floor")
        out_q.index_copy_(0, at[slot], q.index_select(0, token))
        out_scales.index_copy_(0, at[slot], scales.index_select(0, token))
        return out_q, out_scales

    def silu(v):
        return v * torch.special.expit(v)

    def weight(q, scales, first, n):
        """Rows first .. first + n of q in 64 bits, block by block of rows; `scales` are theirs."""
        out = q[first:first + n].double()
        per = torch.arange(q.shape[1], device=DEV) // BLOCK
        for b in range(scales.shape[0]):
            out[b * BLOCK:(b + 1) * BLOCK] *= scales[b].double()[per]
        return out

    if c["op"] == "matmul":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        starts, n = s["starts"].to(torch.int64), c["out"]
        which = torch.bucketize(torch.arange(s["routed"], device=DEV), starts[1:], right=True)
        per = torch.arange(c["depth"], device=DEV) // BLOCK
        for a in range(int((s["expert_ids"] >= 0).sum())):
            rows = (which == a).nonzero().view(-1)
            e = int(s["expert_ids"][a])
            left = s["a"][int(rows[0]):int(rows[-1]) + 1].double()
            if c["type"] == "bf16":
                right = [s["w"][e][first:first + n].double() for first in range(0, s["w"].shape[1], n)]
            else:
                left = left * s["a_scales"][rows].double().index_select(1, per)
                right = [weight(s["w"][e], s["w_scales"][e][i * _blocks(n):(i + 1) * _blocks(n)], i * n, n)
                         for i in range(2 if c["swiglu"] else 1)]
            y = torch.mm(left, right[0].t())
            out.index_copy_(0, rows, silu(y) * torch.mm(left, right[1].t()) if c["swiglu"] else y)
        return out

    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    blocks = _blocks(c["inter"])
    for e in range(c["experts"]):
        token, choice = (s["ids"] == e).nonzero(as_tuple=True)
        if token.numel() == 0:
            continue
        gate = weight(s["w_gate_up"][e], s["gate_up_scales"][e][:blocks], 0, c["inter"])
        up = weight(s["w_gate_up"][e], s["gate_up_scales"][e][blocks:], c["inter"], c["inter"])
        down = weight(s["w_down"][e], s["down_scales"][e], 0, c["hidden"])
        x = s["x"][token].double()
        h = silu(torch.mm(x, gate.t())) * torch.mm(x, up.t())
        share = s["router_weights"][token, choice].double().unsqueeze(1)
        out.index_add_(0, token, share * torch.mm(h, down.t()))
    return out
