"""Every form that the grouped int8 product and the row quantisation take, on
the GPU, against the definition in 64 bits.

The product's sums are exact, so its plain form is compared bit for bit; with
SwiGLU half a bf16 step (2^-8) and the fp32 evaluation count (2^-17, as in
test_gpu_experts).  Quantisation is exact by its definition."""
import numpy as np
import pytest
import torch

from tests.gpu_common import gpu_available, u16
from tests.test_gpu_experts import DEV, SILU, TINY, _csr, dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

mod = pytest.importorskip("expert_grouping_dispatch_amd") if gpu_available() else None


def bytes_of(g, *shape):
    out = torch.empty(shape, dtype=torch.int8, device=DEV)
    flat, step = out.view(-1), 1 << 28
    for at in range(0, flat.numel(), step):
        n = min(step, flat.numel() - at)
        flat[at:at + n] = torch.randint(-128, 128, (n,), generator=g, device=DEV, dtype=torch.int8)
    return out


def check_product(counts, spare, depth, n, swiglu, seed):
    print("[matmul form]", len(counts), sum(counts), depth, n, swiglu, flush=True)
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, wide, v = sum(counts) + spare, n * (2 if swiglu else 1), sum(counts)
    a, w = bytes_of(g, rows, depth), bytes_of(g, len(counts), wide, depth)
    sa = (0.5 + torch.rand(rows, generator=g, device=DEV)) / 73
    sw = (0.5 + torch.rand((len(counts), wide), generator=g, device=DEV)) / (73 * depth ** 0.5)
    sa[v:] = float("nan")
    starts, ids = _csr(counts)
    out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
    mod.moe_expert_matmul_i8(a, sa, dev(starts.view(np.int32)).view(torch.uint32), dev(ids), w, sw, out,
                             flags=mod.MATMUL_SWIGLU if swiglu else 0)
    assert (out[v:] == 7.0).all()
    at = 0
    for e, c in enumerate(counts):
        if c == 0:
            continue
        sums = torch.mm(a[at:at + c].double(), w[e].double().t()).float()  # below 2^53: exact, then one rounding
        y = sums * sa[at:at + c, None] * sw[e]
        got = out[at:at + c]
        if swiglu:
            gate, up = y[:, :n].double(), y[:, n:].double()
            want = gate * torch.special.expit(gate) * up
            bad = (got.double() - want).abs() > SILU * want.abs() + TINY
            assert not bad.any(), (e, c, bad.nonzero()[:4].tolist())
        else:
            np.testing.assert_array_equal(u16(got), u16(y.to(torch.bfloat16)), err_msg=f"expert {e} of {c} rows")
        at += c


MIXED = [300, 100, 256, 70, 129, 513, 66, 200]  # tiles of 65..128 and of 129..256 rows beside each other

FORMS = [
    # rows of each expert, spare rows, depth, output channels
    (MIXED * 8, 3, 256, 1024),                         # 352 tiles (twice that with SwiGLU) of two steps of k
    (MIXED * 8, 3, 384, 1024),                         # of three
    (MIXED * 8, 0, 1024, 2064),                        # 792 and more, of eight; a last column tile of 16 channels
    (MIXED * 8, 0, 128, 1040),                         # of one
    (MIXED * 8, 5, 272, 1024),                         # rows that end inside a step, three steps
    (MIXED * 6, 5, 1040, 1296),                        # nine
    ([65, 128, 0, 127, 66] * 16, 1, 640, 2048),        # tiles of up to 128 rows only
    ([129, 256, 257, 0, 500] * 12, 1, 640, 2048),      # of more only, but for the last rows of a group
    (list(range(0, 65)) * 2, 2, 1024, 1024),           # 0 to 64 rows an expert, through LDS
    (list(range(0, 65)) * 2, 2, 384, 1024),
    (list(range(64, 0, -1)), 1, 1040, 1296),
    ([20, 64, 300, 1, 33, 90] * 12, 7, 768, 1024),     # both sizes in one call
    ([3, 64, 17], 40, 4096, 512),                      # few workgroups
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("case", range(len(FORMS)))
def test_matmul_forms(case, swiglu):
    counts, spare, depth, n = FORMS[case]
    check_product(counts, spare, depth, n, swiglu, case)


@pytest.mark.parametrize("swiglu", [False, True])
def test_matmul_with_weights_beyond_2_gib(swiglu):
    """Byte offsets of the weights pass 31 bits, and 32 with the last experts; small and large groups lie there."""
    counts = [5, 70, 0, 300, 64, 2] * 6 + [33, 129, 1, 260]
    check_product(counts, 2, 8208, 8192 if not swiglu else 4096, swiglu, 50)
    check_product([1] * 66, 0, 8192, 8192 if not swiglu else 4096, swiglu, 51)


@pytest.mark.parametrize("h", [4096, 16000, 28672, 40000])
def test_quantize_buffers_larger_than_the_caches(h):
    """Rows of each length class, with a count below the buffer's rows: bit-exact, the rows behind untouched."""
    n = (256 << 20) // (3 * h) + 8
    real = n - 5
    print("[quantize large]", n, h, flush=True)
    g = torch.Generator(device=DEV).manual_seed(h)
    x = torch.randn((n, h), generator=g, device=DEV, dtype=torch.bfloat16)
    x *= torch.exp2(torch.randint(-40, 40, (n, 1), generator=g, device=DEV).float()).to(torch.bfloat16)
    x[1] = 0
    q = torch.full((n, h), 77, dtype=torch.int8, device=DEV)
    s = torch.full((n,), -3.0, device=DEV)
    mod.moe_quantize_i8(x, q, s, dev(np.array([real], np.int32)).view(torch.uint32))
    a = x.abs().amax(1).double().clamp(min=2.0 ** -118)
    want = torch.round(x.float() * (127 / a).float()[:, None]).to(torch.int8)
    assert torch.equal(q[:real], want[:real]) and torch.equal(s[:real], (a / 127).float()[:real])
    assert (q[real:] == 77).all() and (s[real:] == -3.0).all()
