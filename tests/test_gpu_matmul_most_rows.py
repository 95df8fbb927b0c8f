"""The grouped products over the largest buffers they take, 2^32 - 2 rows of 16
values to 16 outputs: small and large groups whose last row is the buffer's
last, and one expert that has all rows.  Row numbers, rounded up to the next
step or tile, pass 32 bits there.  (bf16 operands and results of that many rows
do not fit the GPU's memory.)"""
import gc

import pytest
import torch

from tests.gpu_common import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

mod = pytest.importorskip("expert_grouping_dispatch_amd") if gpu_available() else None
DEV = "cuda"
ROWS = 2 ** 32 - 2


def _u32(values):
    return torch.tensor(values, dtype=torch.int64, device=DEV).to(torch.uint32)


@pytest.mark.parametrize("kind", ["f8", "i8"])
def test_groups_that_end_with_the_largest_buffer(kind):
    gc.collect()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 240e9:
        pytest.skip("needs 240 GB of free GPU memory")
    f8 = kind == "f8"
    one = 0x38 if f8 else 1  # the value 1 in either type
    a = torch.empty((ROWS, 16), dtype=torch.uint8, device=DEV)
    scales = torch.empty((ROWS, 1) if f8 else ROWS, device=DEV)
    w = torch.full((256, 16, 16), one, dtype=torch.uint8, device=DEV)
    w_scales = torch.ones((256, 1, 1) if f8 else (256, 16), device=DEV)
    out = torch.empty((ROWS, 16), dtype=torch.bfloat16, device=DEV)
    typed = (lambda t: t.view(torch.float8_e4m3fn)) if f8 else (lambda t: t.view(torch.int8))
    call = mod.moe_expert_matmul_f8 if f8 else mod.moe_expert_matmul_i8

    def run(starts, ids, e):
        print("[most rows]", kind, starts, e, flush=True)
        starts, ids = starts + [ROWS] * (e + 1 - len(starts)), ids + [-1] * (e - len(ids))
        call(typed(a), scales, _u32(starts), torch.tensor(ids, dtype=torch.int32, device=DEV), typed(w[:e]), w_scales[:e],
             out)
        torch.cuda.synchronize()

    for e, last in [(e, last) for e in (2, 256) for last in (10, 64, 65, 300)]:  # few rows straight to registers, as strips
        before = ROWS - last  # rows of an id out of range, which are not read
        for t in (a[:4096], a[before - 512:before]):
            t.fill_(0x7F)
        out[:4096], out[before - 512:before], out[before:] = 7.0, 7.0, -1.0
        a[before:], scales[before:] = one, 1.0
        row = torch.arange(1, last + 1, device=DEV).float()  # exact in bf16 up to 256; 257 and on round
        scales[before:] = row[:, None] if f8 else row
        run([0, before, ROWS], [-1, 0], e)
        want = (16 * row).to(torch.bfloat16)[:, None].expand(last, 16)
        assert torch.equal(out[before:], want), last
        assert (out[:4096] == 7.0).all() and (out[before - 512:before] == 7.0).all(), last
    a.fill_(one), scales.fill_(1.0), out.fill_(7.0)
    run([0, ROWS], [0], 2)
    step = 2 ** 28
    for at in range(0, ROWS, step):
        assert (out[at:at + step] == 16.0).all(), at
    del a, scales, out
    gc.collect()
    torch.cuda.empty_cache()
