"""Sizes of tensors that the C entry points take as 32 bits: rows longer than
that are refused, and no shorter ones are made of them."""
import pytest
import torch

from tests.gpu_common import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

mod = pytest.importorskip("expert_grouping_dispatch_amd") if gpu_available() else None
DEV = "cuda"
H = 2 ** 32 + 16


def test_rows_longer_than_32_bits_are_refused():
    x = torch.empty((1, H), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((1, H), dtype=torch.uint8, device=DEV)
    s = torch.full((1, -(-H // 128)), -3.0, device=DEV)
    place = torch.zeros(1, dtype=torch.int32, device=DEV).view(torch.uint32)
    head, f8, i8 = q[0, :64], q.view(torch.float8_e4m3fn), q.view(torch.int8)
    x[0, :64], head[:] = 1.0, 77
    weight = torch.ones(1, device=DEV)
    out = torch.zeros((1, 64), dtype=torch.bfloat16, device=DEV)
    starts, ids = torch.tensor([0, 1], dtype=torch.int32, device=DEV).view(torch.uint32), place.view(torch.int32)
    for call in (lambda: mod.moe_quantize_f8(x, f8, s), lambda: mod.moe_dispatch_f8(x, 1, place, f8, s),
                 lambda: mod.moe_quantize_i8(x, i8, s[0, :1]), lambda: mod.moe_dispatch_i8(x, 1, place, i8, s[0, :1]),
                 lambda: mod.moe_dispatch(x, 1, place, x), lambda: mod.moe_combine(x, weight, place, 1, x),
                 lambda: mod.moe_combine_epilogue(x, weight, place, 1, x),
                 lambda: mod.moe_dispatch_mxfp4(x, 1, place, q[:, :H // 2], torch.empty((1, H // 32), dtype=torch.uint8, device=DEV)),
                 lambda: mod.moe_expert_matmul(x, starts, ids, x.view(1, 1, H), out[:, :1]),
                 lambda: mod.moe_expert_matmul_f8(f8, s, starts, ids, f8.view(1, 1, H), s.view(1, 1, -1), out[:, :1])):
        with pytest.raises(ValueError, match=f"^{H} does not fit 32 bits"):
            call()
    torch.cuda.synchronize()
    assert (head == 77).all() and (s == -3.0).all() and (x[0, :64] == 1.0).all()
