"""The whole layer for a few tokens on e4m3 weights with a scale for each block
of 128 x 128, on the GPU, in every form that its products take.

On whole numbers and powers of two no rounding happens before the output's own:
results are compared bit for bit, and need up to 12 bits of the activations
between the products.  On normal values the oracle's bound of the layer holds: a
block's sum times its scale is added in one rounding, so a product passes
through fewer roundings than the sum has products."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_common import gpu_available, u16
from tests.test_gpu_experts import LAYERS, _ids, _layer_call, dev, f64
from tests.test_gpu_layer_forms import SHARED, SIXTEEN_BITS, _counted

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

mod = pytest.importorskip("expert_grouping_dispatch_amd") if gpu_available() else None
DEV = "cuda"
F8 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // 128)


def per_value(scales, n, k, halves=1):
    """[halves * n, k] of one expert's scales."""
    rows = scales.double().view(halves, blocks(n), -1)[:, torch.arange(n, device=DEV) // 128].reshape(halves * n, -1)
    return rows[:, torch.arange(k, device=DEV) // 128]


def whole_layer(n, k, e, h, i, ids, seed):
    """(arguments of _layer_call, the exact output).  gate is 32, so silu(gate) is 32 to the last bit of fp32.  up is
    a product of an odd number below 256 and one below 16, plus small numbers of every further column of x, so that
    an activation read from the wrong place shows, times powers of two.  About twelve values of each row of w_down
    are not 0.  Sums of magnitudes stay below 2^24 of the least step, so every partial sum is exact in fp32."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def ints(lo, hi, *shape, dtype=torch.int8):
        return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=dtype)

    x = torch.where(torch.rand((n, h), generator=g, device=DEV) < min(1.0, 16 / h), ints(-1, 2, n, h), 0).float()
    x[:, 0], x[:, 1] = 1, 2.0 * ints(0, 128, n, dtype=torch.int16) + 1
    sg = torch.exp2(ints(-1, 2, e, 2 * blocks(i), blocks(h)).float())
    sd = torch.exp2(ints(-1, 2, e, blocks(h), blocks(i)).float())
    wgu, wd = (torch.empty(s, dtype=F8, device=DEV) for s in ((e, 2 * i, h), (e, h, i)))
    rw = torch.exp2(ints(-1, 1, n, k).float())
    want = torch.zeros((n, h), dtype=torch.float64, device=DEV)
    total = torch.zeros((n, h), dtype=torch.float64, device=DEV)
    choice = torch.from_numpy(ids.astype(np.int64)).to(DEV)
    for a in range(e):
        v, per = torch.zeros((2 * i, h), device=DEV), per_value(sg[a], i, h, 2)
        v[:i, 0] = 32 / per[:i, 0].float()
        v[i:] = ints(-1, 2, i, h)
        v[i:, 1] = 2.0 * ints(-8, 8, i) + 1
        wgu[a] = v.to(F8)
        d = torch.where(torch.rand((h, i), generator=g, device=DEV) < 12 / i, ints(-1, 2, h, i), 0).float()
        wd[a] = d.to(F8)
        t, j = (choice == a).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        both = torch.mm(x[t].double(), (v.double() * per).t())
        assert (both[:, :i] == 32).all()
        act, down = 32 * both[:, i:], (d.double() * per_value(sd[a], h, i)).t()
        share = rw[t, j].double().unsqueeze(1)
        want.index_add_(0, t, share * torch.mm(act, down))
        total.index_add_(0, t, share * torch.mm(act.abs(), down.abs()))
    assert total.max() < 4 * 2 ** 24  # steps of 32 / 2 from up's scale, / 2 from down's, / 2 from the router's
    return (x.to(torch.bfloat16), ids, rw.cpu().numpy(), wgu, wd, sg, sd), want.float().to(torch.bfloat16)


def check(n, k, e, h, i, ids, seed, **more):
    print("[layer f8]", n, k, e, h, i, flush=True)
    args, want = whole_layer(n, k, e, h, i, ids, seed)
    np.testing.assert_array_equal(u16(_layer_call(*args, **more)), u16(want))


@pytest.mark.parametrize("case", range(len(LAYERS)))
def test_layer_on_whole_numbers(case):
    n, k, e, h, i, kind = LAYERS[case]
    check(n, k, e, h, i, _ids(np.random.default_rng(600 + case), n, k, e, kind), 600 + case, ids64=case % 2 == 1)


@pytest.mark.parametrize("case", range(len(SIXTEEN_BITS)))
def test_layer_on_whole_numbers_more_slots(case):
    n, k, e, h, i, kind = SIXTEEN_BITS[case]
    check(n, k, e, h, i, _ids(np.random.default_rng(630 + case), n, k, e, kind), 630 + case)


@pytest.mark.parametrize("case", range(len(SHARED)))
def test_layer_with_many_slots_on_an_expert(case):
    counts, k, h, i = SHARED[case]
    ids = _counted(counts, k, 660 + case)
    check(len(ids), k, len(counts), h, i, ids, 660 + case)


@pytest.mark.parametrize("n, k, e, h, i", [(3, 2, 9, 7168, 2048), (40, 8, 64, 7168, 400), (9, 1, 1, 5136, 1296),
                                           (1, 2, 4, 4096, 14336), (20, 2, 2, 8192, 1408)])
def test_layer_of_wide_rows(n, k, e, h, i):
    """28, 20 or 32 channels a workgroup, so that some have rows in two blocks."""
    check(n, k, e, h, i, _ids(np.random.default_rng(n), n, k, e, "distinct"), 690 + n)


@pytest.mark.parametrize("case", range(len(LAYERS)))
def test_layer_against_the_bound(case):
    """Weights are every finite code, unused experts NaN, tokens without a choice NaN."""
    n, k, e, h, i, kind = LAYERS[case]
    print("[layer f8 bound]", case, flush=True)
    g = np.random.default_rng(700 + case)
    ids, rw = _ids(g, n, k, e, kind), g.random((n, k)).astype(np.float32)
    x = dev(g.standard_normal((n, h)).astype(np.float32), torch.bfloat16)
    x[torch.from_numpy(((ids < 0) | (ids >= e)).all(1))] = float("nan")
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    qgu, qd = codes[g.integers(0, 254, (e, 2 * i, h))], codes[g.integers(0, 254, (e, h, i))]
    sg = ((0.5 + g.random((e, 2 * blocks(i), blocks(h)))) / (120 * h ** 0.5)).astype(np.float32)
    sd = ((0.5 + g.random((e, blocks(h), blocks(i)))) / (120 * i ** 0.5)).astype(np.float32)
    values = oracle.e4m3_values()
    fgu = np.stack([oracle.block_weights(values[qgu[a]], sg[a], 2) for a in range(e)])
    fd = np.stack([oracle.block_weights(values[qd[a]], sd[a]) for a in range(e)])
    unused = sorted(set(range(e)) - set(ids.reshape(-1).tolist()))
    qgu[unused], qd[unused], sg[unused], sd[unused] = 0x7F, 0xFF, np.nan, np.nan
    out = _layer_call(x, ids, rw, dev(qgu).view(F8), dev(qd).view(F8), dev(sg), dev(sd), ids64=case % 2 == 0)
    want, bound = oracle.layer_few(f64(x), ids, rw, fgu, fd)
    bad = ~(np.abs(f64(out) - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], f64(out)[bad][:4], want[bad][:4], bound[bad][:4])


def test_a_tokens_result_does_not_depend_on_the_padding():
    n, k, e, h, i = 40, 3, 12, 272, 144
    ids = _ids(np.random.default_rng(7), n, k, e, "distinct")
    args, want = whole_layer(n, k, e, h, i, ids, 7)
    x, rw = args[0], args[2]
    for rows in (n, 300, 600):
        wide_x = torch.full((rows, h), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide_x[:n] = x
        wide_ids, wide_rw = np.zeros((rows, k), np.int32), np.ones((rows, k), np.float32)
        wide_ids[:n], wide_rw[:n] = ids, rw
        out = _layer_call(wide_x, wide_ids, wide_rw, *args[3:], count=n)
        np.testing.assert_array_equal(u16(out[:n]), u16(want))
        assert not u16(out[n:]).any()


@pytest.mark.parametrize("n, k, e, h, i", [(1, 2, 8, 4096, 1040), (12, 4, 9, 272, 400), (200, 2, 3, 144, 272)])
def test_layer_captured_and_with_the_least_alignment(n, k, e, h, i):
    """Scales that begin at 4 bytes; two captured calls with workspaces of their own, replayed at once on two streams
    with other maps and other counts than the captured ones."""
    steps = []
    for turn in range(2):
        per_map = []
        for m in range(3):
            ids = _ids(np.random.default_rng(10 * turn + m), n, k, e, "distinct")
            args, _ = whole_layer(n, k, e, h, i, ids, 40 + turn)  # the same weights, other maps
            per_map.append((ids, args, [_layer_call(*args, count=c) for c in (n, n // 2)]))
        sg, sd = per_map[0][1][5:]
        moved = []
        for t in (sg, sd):
            room = torch.full((t.numel() + 2,), float("nan"), device=DEV)
            room[1:-1] = t.reshape(-1)
            moved.append(room[1:-1].view(t.shape))
        steps.append((per_map, moved))
    graphs = []
    for per_map, moved in steps:
        _, args, _ = per_map[0]
        x, rw = args[0].clone(), dev(args[2])
        ids, count = dev(per_map[0][0]), dev(np.array([n], np.int32))
        out, space = torch.zeros_like(x), mod.alloc_layer_few(n, k, i, DEV)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            mod.moe_layer_few(x, ids, rw, args[3], args[4], out, space, gate_up_scales=moved[0], down_scales=moved[1],
                              real_token_count=count)
        graphs.append((graph, x, ids, rw, count, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for replay in range(6):
        for (per_map, _), (graph, x, ids, rw, count, out) in zip(steps, graphs):
            new_ids, args, _ = per_map[replay % 3]
            x.copy_(args[0]), ids.copy_(dev(new_ids)), rw.copy_(dev(args[2]))
            count.fill_((n, n // 2)[replay % 2])
            out.fill_(7.0)
        torch.cuda.synchronize()
        for stream, g in zip(streams, graphs):
            with torch.cuda.stream(stream):
                g[0].replay()
        torch.cuda.synchronize()
        for (per_map, _), g in zip(steps, graphs):
            np.testing.assert_array_equal(u16(g[5]), u16(per_map[replay % 3][2][replay % 2]))


def test_layer_with_weights_beyond_4_gib():
    """Byte offsets of both weights pass 31 bits, and 32 in the first product."""
    n, k, e, h, i = 40, 4, 68, 8192, 4096
    ids = _ids(np.random.default_rng(8), n, k, e, "distinct")
    ids[0, 0], ids[1] = e - 1, [e - 2, 0, e - 3, 1]
    check(n, k, e, h, i, ids, 720)


def test_layer_agrees_with_the_grouped_calls():
    """The same weights through moe_expert_matmul_f8 on activations that e4m3 holds exactly: whole numbers up to 15
    of scale 1 in the first product; the second product's activations are held in e4m3 there, to half a step."""
    n, k, e, h, i = 150, 2, 4, 272, 400
    g = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randint(-15, 16, (n, h), generator=g, device=DEV).float()
    ids = _ids(np.random.default_rng(11), n, k, e, "distinct")
    wgu = (torch.randn((e, 2 * i, h), generator=g, device=DEV) * 105).clamp(-448, 448).to(F8)
    wd = (torch.randn((e, h, i), generator=g, device=DEV) * 105).clamp(-448, 448).to(F8)
    sg = (0.5 + torch.rand((e, 2 * blocks(i), blocks(h)), generator=g, device=DEV)) / (105 * 8 * h ** 0.5)
    sd = (0.5 + torch.rand((e, blocks(h), blocks(i)), generator=g, device=DEV)) / (105 * i ** 0.5)
    rw = np.random.default_rng(12).random((n, k)).astype(np.float32)
    few = f64(_layer_call(x.to(torch.bfloat16), ids, rw, wgu, wd, sg, sd))
    idx = mod.alloc_indices(n * k, e, DEV)
    mod.moe_create_indices(dev(ids), e, idx["token_expert_order"], idx["expert_start_indices"],
                           idx["restore_token_order"], idx["expert_ids"], idx["expert_usage_stats"], idx["workspace"])
    order = idx["token_expert_order"].to(torch.int64)
    a, ones = x[order // k].to(F8), torch.ones((n * k, blocks(h)), device=DEV)
    act = torch.zeros((n * k, i), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((n * k, h), dtype=torch.bfloat16, device=DEV)
    starts, active = idx["expert_start_indices"], idx["expert_ids"]
    mod.moe_expert_matmul_f8(a, ones, starts, active, wgu, sg, act, flags=mod.MATMUL_SWIGLU)
    q, s = mod.alloc_quantized_f8(n * k, i, DEV)
    mod.moe_quantize_f8(act, q, s, row_count=starts[-1:])
    mod.moe_expert_matmul_f8(q, s, starts, active, wd, sd, y)
    out = torch.zeros((n, h), dtype=torch.bfloat16, device=DEV)
    mod.moe_combine(y, dev(rw), idx["restore_token_order"], k, out)
    # half a step of e4m3 on each of 400 activations: the errors' root mean square is at most 2^-4 of the result's
    d = f64(out) - few
    assert np.sqrt((d ** 2).mean()) < 2.0 ** -4 * np.sqrt((few ** 2).mean())
