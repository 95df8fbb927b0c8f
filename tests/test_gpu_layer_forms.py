"""Every form that moe_layer_few's products take, on the GPU.

The forms follow from the slots an expert has, the slots of the map, the widths
and the number of workgroups.  Weights and activations are whole numbers chosen
so that no rounding happens before the output's own: results are compared bit
for bit, and need all 14 bits of the activations between the products."""
import numpy as np
import pytest
import torch

from tests.gpu_common import gpu_available, u16
from tests.test_gpu_experts import DEV, _ids, _layer_call

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def whole_layer(n, k, e, h, i, ids, weights, seed):
    """(arguments of _layer_call, the exact output).

    gate is 32, so silu(gate) is 32 to the last bit of fp32.  up is a product of two odd numbers below 128, up to 14
    bits, plus a small number of every further column of x, so that an activation read from the wrong place shows.
    About twelve values of each row of w_down are not 0.  Sums of the magnitudes stay below 2^24 steps of 16 (32 times
    the router weights' 1/2), so every partial sum is exact in fp32 whatever its order."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def ints(lo, hi, *shape, dtype=torch.int8):
        return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=dtype)

    x = torch.where(torch.rand((n, h), generator=g, device=DEV) < min(1.0, 16 / h), ints(-1, 2, n, h), 0).to(torch.int8)
    x[:, 0], x[:, 1] = 1, 2 * ints(0, 64, n) + 1
    wgu = torch.empty((e, 2 * i, h), dtype=torch.int8, device=DEV)
    for a in range(e):
        wgu[a, :i], wgu[a, i:] = 0, ints(-1, 2, i, h)
        wgu[a, :i, 0] = 32
        wgu[a, i:, 1] = 2 * ints(-64, 64, i) + 1
    wd = torch.empty((e, h, i), dtype=torch.int8, device=DEV)
    for a in range(e):
        wd[a] = torch.where(torch.rand((h, i), generator=g, device=DEV) < 12 / i, ints(-1, 2, h, i), 0)
    rw = torch.exp2(ints(-1, 1, n, k).float())
    want = torch.zeros((n, h), dtype=torch.float64, device=DEV)
    total = torch.zeros((n, h), dtype=torch.float64, device=DEV)
    choice = torch.from_numpy(ids.astype(np.int64)).to(DEV)
    for a in range(e):
        t, j = (choice == a).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        xe = x[t].double()
        assert (torch.mm(xe, wgu[a, :i].double().t()) == 32).all()
        act = 32 * torch.mm(xe, wgu[a, i:].double().t())
        assert act.abs().max() < 32 * 2 ** 15
        down = wd[a].double().t()
        share = rw[t, j].double().unsqueeze(1)
        want.index_add_(0, t, share * torch.mm(act, down))
        total.index_add_(0, t, share * torch.mm(act.abs(), down.abs()))
    assert total.max() < 16 * 2 ** 24
    one = torch.int8 if weights == "int8" else torch.bfloat16
    scales = (None, None) if weights == "bf16" else (torch.ones((e, 2 * i), device=DEV), torch.ones((e, h), device=DEV))
    return (x.to(torch.bfloat16), ids, rw.cpu().numpy(), wgu.to(one), wd.to(one), *scales), want.float().to(torch.bfloat16)


def check(n, k, e, h, i, ids, weights, seed, **more):
    print("[layer form]", n, k, e, h, i, weights, flush=True)
    args, want = whole_layer(n, k, e, h, i, ids, weights, seed)
    np.testing.assert_array_equal(u16(_layer_call(*args, **more)), u16(want))


SIXTEEN_BITS = [
    # rows, top_k, experts, hidden, inter, ids: slots an expert has, or of the map, above the few that fit beside h
    (12, 1, 3, 144, 80, "one"),              # 12 slots on an expert, one row tile
    (16, 1, 2, 6160, 144, "one"),            # 16, two row tiles
    (9, 1, 2, 48, 1552, "one"),              # long rows
    (70, 3, 5, 144, 80, "one"),              # 210
    (45, 1, 2, 6160, 80, "one"),
    (20, 1, 2, 64, 1296, "one"),
    (256, 8, 256, 48, 32, "distinct"),       # 2048 slots of the map
    (130, 8, 300, 6144, 48, "distinct"),
    (600, 1, 200, 64, 1296, "distinct"),
    (72, 8, 160, 4112, 1296, "distinct"),    # long rows in two row tiles
    (300, 5, 3, 2080, 144, "mixed"),
]


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("case", range(len(SIXTEEN_BITS)))
def test_layer_keeps_sixteen_bits_between_the_products(case, weights):
    n, k, e, h, i, kind = SIXTEEN_BITS[case]
    check(n, k, e, h, i, _ids(np.random.default_rng(300 + case), n, k, e, kind), weights, 300 + case)


def test_a_tokens_result_does_not_depend_on_the_padding():
    """The same 40 tokens in a map of 40, 300 and 600 rows, on experts that 5 to 16 of their slots share."""
    n, k, e, h, i = 40, 3, 12, 272, 144
    ids = _ids(np.random.default_rng(7), n, k, e, "distinct")
    args, want = whole_layer(n, k, e, h, i, ids, "bf16", 7)
    x, rw = args[0], args[2]
    for rows in (n, 300, 600):
        wide_x = torch.full((rows, h), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide_x[:n] = x
        wide_ids, wide_rw = np.zeros((rows, k), np.int32), np.ones((rows, k), np.float32)
        wide_ids[:n], wide_rw[:n] = ids, rw
        out = _layer_call(wide_x, wide_ids, wide_rw, *args[3:], count=n)
        np.testing.assert_array_equal(u16(out[:n]), u16(want))
        assert not u16(out[n:]).any()
