"""What is measured of the expert products: int8 dispatch, row quantisation, the
grouped int8 product and the whole layer for a few tokens.

``run`` computes a case in plain torch operations in 32 bits where ``own`` is
false, and through the framework's entry points where it is true.  ``exact``
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- cases ------------------------------------------------------------------------------------------------


def listed():
    return [
        # int8 dispatch: the tiny workload, a captured decode batch with padding rows, a skewed prefill
        dict(name="dispatch tiny", op="dispatch", rows=64, real=64, hidden=256, experts=8, top_k=2, routing="uniform"),
        dict(name="dispatch decode", op="dispatch", rows=256, real=97, hidden=7168, experts=256, top_k=8,
             routing="uniform"),
        dict(name="dispatch prefill", op="dispatch", rows=4096, real=4096, hidden=7168, experts=256, top_k=8,
             routing="zipf"),
        # activations between the two products: a decode batch in its padded buffer, a long prefill with wide experts
        dict(name="quantize decode", op="quantize", rows=2048, real=776, hidden=2048),
        dict(name="quantize prefill", op="quantize", rows=16384, real=14000, hidden=14336),
        # grouped product: a decode batch spread over many experts, a prefill over few and wide ones (both the first
        # product with its SwiGLU), and the second product of a skewed prefill and of the largest batch
        dict(name="matmul decode swiglu", op="matmul", rows=256, real=97, experts=256, top_k=8, routing="uniform",
             depth=7168, out=2048, swiglu=True),
        dict(name="matmul prefill swiglu", op="matmul", rows=8192, real=7000, experts=8, top_k=2, routing="uniform",
             depth=4096, out=14336, swiglu=True),
        dict(name="matmul prefill down", op="matmul", rows=4096, real=4096, experts=256, top_k=8, routing="zipf",
             depth=2048, out=7168, swiglu=False),
        dict(name="matmul stress down", op="matmul", rows=65536, real=61440, experts=256, top_k=8, routing="hotcold",
             depth=2048, out=7168, swiglu=False),
        # whole layer: one token, a small odd batch over small experts, a captured decode batch with int8 weights
        dict(name="layer one token", op="layer", rows=1, real=1, hidden=4096, inter=14336, experts=8, top_k=2,
             routing="uniform", weights="bf16"),
        dict(name="layer odd", op="layer", rows=24, real=13, hidden=1040, inter=528, experts=24, top_k=4,
             routing="uniform", weights="bf16"),
        dict(name="layer decode int8", op="layer", rows=256, real=97, hidden=7168, inter=2048, experts=256, top_k=8,
             routing="uniform", weights="int8"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    """A row length: a multiple of 16, spread over the logarithm."""
    return 16 * max(1, _spread(rng, lo, hi) // 16)


def draw(rng):
    while True:
        op = rng.choice(("dispatch", "quantize", "matmul", "matmul", "layer", "layer"))
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
            c.update(depth=_wide(rng, 64, 8192), out=_wide(rng, 64, 8192), swiglu=rng.random() < 0.5)
            wide = c["out"] * (2 if c["swiglu"] else 1)
            if experts * c["depth"] * wide <= 3.7e9 and slots * c["depth"] * wide <= 1e12:
                return c
        else:
            c.update(hidden=_wide(rng, 256, 8192), inter=_wide(rng, 128, 8192), weights=rng.choice(("bf16", "int8")))
            if experts * c["hidden"] * c["inter"] <= 1.25e9:
                return c


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
        return {"bytes": c["real"] * (3 * c["hidden"] + 4) or 4, "flops": 3 * c["real"] * c["hidden"]}
    slots = c["real"] * c["top_k"]
    if c["op"] == "dispatch":
        return {"bytes": 2 * c["real"] * c["hidden"] + slots * (c["hidden"] + 4) + 4 * c["rows"] * c["top_k"],
                "flops": 3 * c["real"] * c["hidden"]}
    if c["op"] == "matmul":
        wide = c["out"] * (2 if c["swiglu"] else 1)
        return {"bytes": slots * (c["depth"] + 4 + 2 * c["out"]) + _active(c) * wide * (c["depth"] + 4),
                "flops": 2 * slots * c["depth"] * wide}
    each = 3 * c["hidden"] * c["inter"]
    if c["weights"] == "bf16":
        each *= 2
    else:
        each += 4 * (2 * c["inter"] + c["hidden"])
    return {"bytes": _active(c) * each + 2 * (c["real"] + c["rows"]) * c["hidden"] + 8 * c["rows"] * c["top_k"],
            "flops": 6 * slots * c["hidden"] * c["inter"]}


# ---- inputs -----------------------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    """Normal values in `dtype`, drawn in pieces; int8 is what 8-bit rows hold: the largest of a few
    thousand values at 127, so about 28 to one standard deviation."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat, step = out.view(-1), 1 << 27
    for at in range(0, flat.numel(), step):
        v = torch.randn(min(step, flat.numel() - at), generator=g, device=DEV)
        flat[at:at + step] = v.mul_(28).round_().clamp_(-127, 127) if dtype == torch.int8 else v.mul_(scale)
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


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=dict(case))
    if c["op"] == "quantize":
        s["x"] = _normal(g, (c["rows"], c["hidden"]), torch.bfloat16)
        s["count"] = torch.tensor([c["real"]], dtype=torch.int64, device=DEV).to(torch.uint32)
        s["out_q"] = torch.zeros((c["rows"], c["hidden"]), dtype=torch.int8, device=DEV)
        s["out_scales"] = torch.zeros(c["rows"], dtype=torch.float32, device=DEV)
        return s
    ids = _routing(c, g)
    slots = ids.numel()
    s.update(_indices(c, ids))
    if c["op"] == "dispatch":
        s["x"] = _normal(g, (c["rows"], c["hidden"]), torch.bfloat16)
        s["out_q"] = torch.zeros((slots, c["hidden"]), dtype=torch.int8, device=DEV)
        s["out_scales"] = torch.zeros(slots, dtype=torch.float32, device=DEV)
    elif c["op"] == "matmul":
        wide = c["out"] * (2 if c["swiglu"] else 1)
        s["a_q"] = _normal(g, (slots, c["depth"]), torch.int8)
        s["a_scales"] = _scales(g, (slots,), 1 / 28)
        s["w_q"] = _normal(g, (c["experts"], wide, c["depth"]), torch.int8)
        s["w_scales"] = _scales(g, (c["experts"], wide), 1 / (28 * c["depth"] ** 0.5))
        s["out"] = torch.zeros((slots, c["out"]), dtype=torch.bfloat16, device=DEV)
    else:
        h, i, e = c["hidden"], c["inter"], c["experts"]
        s["ids"] = ids
        s["x"] = _normal(g, (c["rows"], h), torch.bfloat16)
        s["router_weights"] = torch.softmax(torch.randn(ids.shape, generator=g, device=DEV), 1)
        if c["weights"] == "int8":
            s["w_gate_up"] = _normal(g, (e, 2 * i, h), torch.int8)
            s["w_down"] = _normal(g, (e, h, i), torch.int8)
            s["gate_up_scales"] = _scales(g, (e, 2 * i), 1 / (28 * h ** 0.5))
            s["down_scales"] = _scales(g, (e, h), 1 / (28 * i ** 0.5))
        else:
            s["w_gate_up"] = _normal(g, (e, 2 * i, h), torch.bfloat16, h ** -0.5)
            s["w_down"] = _normal(g, (e, h, i), torch.bfloat16, i ** -0.5)
            s["gate_up_scales"] = s["down_scales"] = None
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
        moe.moe_quantize_i8(s["x"], s["out_q"], s["out_scales"], row_count=s["count"])
        return s["out_q"], s["out_scales"]
    if op == "dispatch":
        moe.moe_dispatch_i8(s["x"], s["case"]["top_k"], s["restore"], s["out_q"], s["out_scales"])
        return s["out_q"], s["out_scales"]
    if op == "matmul":
        moe.moe_expert_matmul_i8(s["a_q"], s["a_scales"], s["starts"], s["expert_ids"], s["w_q"], s["w_scales"],
                                 s["out"], flags=moe.MATMUL_SWIGLU if s["case"]["swiglu"] else 0)
        return s["out"]
    moe.moe_layer_few(s["x"], s["ids"], s["router_weights"], s["w_gate_up"], s["w_down"], s["out"], s["workspace"],
                      gate_up_scales=s["gate_up_scales"], down_scales=s["down_scales"])
    return s["out"]


def _quantized(x):
    """Rows to int8: the divisions in 64 bits and rounded once, the product with the inverse rounded to 32 bits
    before it is rounded to the nearest whole number, ties to the even one, as the format is defined."""
    x = x.float()
    largest = x.abs().amax(1).clamp(min=2.0 ** -118).double()
    q = torch.round(x * (127.0 / largest).float()[:, None])
    return q.to(torch.int8), (largest / 127.0).float()


def _silu_times(gate, up):
    return gate / (1 + torch.exp(-gate)) * up


def _products(s):
    n = s["case"]["out"]
    out = torch.zeros_like(s["out"])
    for e, lo, hi in s["groups"]:
        y = s["a_q"][lo:hi].float() @ s["w_q"][e].float().t()
        y = y * s["a_scales"][lo:hi, None] * s["w_scales"][e]
        out[lo:hi] = _silu_times(y[:, :n], y[:, n:]) if s["case"]["swiglu"] else y
    return out


def _layer(s):
    c = s["case"]
    k, i = c["top_k"], c["inter"]
    y = torch.zeros((c["rows"] * k, c["hidden"]), device=DEV)
    for e, lo, hi in s["groups"]:
        slots = s["order"][lo:hi]
        t = s["x"][slots // k].float() @ s["w_gate_up"][e].float().t()
        if s["gate_up_scales"] is not None:
            t = t * s["gate_up_scales"][e]
        t = _silu_times(t[:, :i], t[:, i:]) @ s["w_down"][e].float().t()
        y[slots] = t if s["down_scales"] is None else t * s["down_scales"][e]
    return (y.view(c["rows"], k, -1) * s["router_weights"][:, :, None]).sum(1).to(torch.bfloat16)


# ---- from the definitions, in 64 bits -----------------------------------------------------------------------


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("quantize", "dispatch"):
        # q = the whole number next to fl32(x * fl32(127 / a)), scale = fl32(a / 127), a = max(|x|, 2^-118)
        x = s["x"].to(torch.float64)
        a = torch.maximum(x.max(1)[0], -x.min(1)[0]).clamp(min=2.0 ** -118).unsqueeze(1)
        inverse = (127 / a).to(torch.float32).to(torch.float64)
        t = (x * inverse).to(torch.float32).to(torch.float64)
        low = torch.floor(t)
        above = t - low
        q = low + ((above > 0.5) | ((above == 0.5) & (low % 2 != 0))).to(torch.float64)
        scales = (a / 127).to(torch.float32).to(torch.float64)[:, 0]
        if c["op"] == "quantize":
            beyond = torch.arange(c["rows"], device=DEV) >= c["real"]
            q[beyond], scales[beyond] = 0, 0
            return q.to(torch.int8), scales
        at = s["restore"].to(torch.int64)
        slot = (at != 0xFFFFFFFF).nonzero().view(-1)
        out_q = torch.zeros(s["out_q"].shape, dtype=torch.int8, device=DEV)
        out_scales = torch.zeros(s["out_scales"].shape, dtype=torch.float64, device=DEV)
        token = torch.div(slot, c["top_k"], rounding_mode="floor")
        out_q.index_copy_(0, at[slot], q.to(torch.int8).index_select(0, token))
        out_scales.index_copy_(0, at[slot], scales.index_select(0, token))
        return out_q, out_scales

    def silu(v):
        return v * torch.special.expit(v)

    if c["op"] == "matmul":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        starts = s["starts"].to(torch.int64)
        which = torch.bucketize(torch.arange(s["routed"], device=DEV), starts[1:], right=True)
        for a in range(int((s["expert_ids"] >= 0).sum())):
            rows = (which == a).nonzero().view(-1)
            e = int(s["expert_ids"][a])
            left = s["a_scales"][rows].double().unsqueeze(1) * s["a_q"][rows].double()
            right = s["w_scales"][e].double().unsqueeze(1) * s["w_q"][e].double()
            if c["swiglu"]:
                y = silu(torch.mm(left, right[:c["out"]].t())) * torch.mm(left, right[c["out"]:].t())
            else:
                y = torch.mm(left, right.t())
            out.index_copy_(0, rows, y)
        return out

    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for e in range(c["experts"]):
        token, choice = (s["ids"] == e).nonzero(as_tuple=True)
        if token.numel() == 0:
            continue
        gate_up, down = s["w_gate_up"][e].double(), s["w_down"][e].double()
        if c["weights"] == "int8":
            gate_up = gate_up * s["gate_up_scales"][e].double().unsqueeze(1)
            down = down * s["down_scales"][e].double().unsqueeze(1)
        x = s["x"][token].double()
        h = silu(torch.mm(x, gate_up[:c["inter"]].t())) * torch.mm(x, gate_up[c["inter"]:].t())
        share = s["router_weights"][token, choice].double().unsqueeze(1)
        out.index_add_(0, token, share * torch.mm(h, down.t()))
    return out
