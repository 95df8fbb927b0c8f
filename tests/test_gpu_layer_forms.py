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


def _counted(counts, k, seed):
    """A map in which expert e has counts[e] slots (a multiple of k in all), in random order."""
    slots = np.repeat(np.arange(len(counts)), counts)
    return np.random.default_rng(seed).permutation(slots).reshape(-1, k).astype(np.int32)


SHARED = [
    # slots of each expert, top_k, hidden, inter: grids that fill the CUs, through LDS 32 or 64 slots at a time
    ([33, 40, 50, 64], 1, 1024, 4096),
    ([33, 40, 51, 64], 2, 1040, 4112),
    ([65, 80, 96, 1], 1, 1024, 4096),
    ([97, 128, 129, 20], 2, 1040, 4096),
    ([300, 64, 32, 200], 4, 144, 4096),
    ([64, 65, 128, 129] * 4, 2, 256, 1040),
    ([2, 5, 8, 9, 16, 17, 32, 33] * 5, 1, 2064, 528),     # every number that changes the second product's form
    ([1, 4, 5, 8, 9, 16, 17, 40] * 3, 2, 4112, 1296),     # with long rows and two row tiles
    ([3, 4, 5, 8, 9, 16, 17, 70], 2, 272, 2064),          # in long rows
    ([1024, 1024], 8, 64, 64),
    ([31, 33, 65, 1, 70], 5, 400, 80),                    # the smallest grids: 16 channels a workgroup
]


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_layer_with_many_slots_on_an_expert(case, weights):
    counts, k, h, i = SHARED[case]
    ids = _counted(counts, k, 400 + case)
    check(len(ids), k, len(counts), h, i, ids, weights, 400 + case)


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("h, i", [(2048, 4096), (4112, 1296)])
def test_layer_with_one_real_token_in_a_large_map(h, i, weights):
    """256 x 8 slots of which one token's are routed, by the count and by the ids."""
    n, k, e = 256, 8, 32
    ids = np.full((n, k), -1, np.int32)
    ids[0] = np.random.default_rng(3).permutation(e)[:k]
    check(n, k, e, h, i, ids, weights, 500)
    args, want = whole_layer(n, k, e, h, i, ids, weights, 501)
    ids[1:] = np.arange(8)
    out = _layer_call(args[0], ids, *args[2:], count=1)
    np.testing.assert_array_equal(u16(out), u16(want))


@pytest.mark.parametrize("weights", ["bf16", "int8"])
def test_layer_with_weights_beyond_2_gib(weights):
    """Byte offsets of both weights pass 31 bits, and 32 in the first product."""
    n, k, e, h, i = 40, 4, 68, 8192, 4096
    ids = _ids(np.random.default_rng(8), n, k, e, "distinct")
    ids[0, 0], ids[1] = e - 1, [e - 2, 0, e - 3, 1]
    check(n, k, e, h, i, ids, weights, 510)
