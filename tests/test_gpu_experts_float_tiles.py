"""The grouped products where a workgroup takes several tiles in turn: their
steps of k, and in e4m3 the groups of four steps' scales, run on from one tile
to the next.  More than 256 tiles, of 65 to 128 and of 129 to 256 rows beside
each other; steps of 128 bytes, odd and even numbers of them, whole and ragged
rows (only of whole ones do the workgroups of an XCD begin in the middle), odd
and even numbers of groups of scales; more rows than the eight tiles that are
taken column by column together.  On whole numbers, bit for bit but for SwiGLU."""
import numpy as np
import pytest

from tests.gpu_common import gpu_available, u16
from tests.test_gpu_experts_float import MIXED, Case, say
from tests.test_gpu_matmul_forms import check_product

import torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

LONG = [2900, 90, 0, 1500, 40, 2100]  # 12, 1, 6 and 9 row tiles
FORMS = [
    # counts per expert, spare rows, depth, weight rows per expert (doubled with SwiGLU)
    (MIXED * 8, 3, 192, 1040),    # bf16: 3 steps
    (MIXED * 8, 3, 384, 1040),    # e4m3: 3 steps, one group of scales
    (MIXED * 8, 0, 448, 1040),    # bf16: 7 steps; e4m3: 4 with a ragged end
    (MIXED * 8, 3, 640, 1040),    # e4m3: 5 steps, two groups
    (MIXED * 8, 0, 896, 1296),    # e4m3: 7 steps
    (MIXED * 8, 5, 1040, 1040),   # e4m3: 9 steps with a ragged end, three groups
    (MIXED * 8, 0, 1152, 1040),   # e4m3: 9 whole steps
    (MIXED * 8, 0, 1088, 1040),   # bf16: 17 whole steps
    (MIXED * 6, 2, 1280, 1552),   # e4m3: 10 steps
    (MIXED * 6, 2, 2176, 1552),   # e4m3: 17 steps, five groups; bf16: 34
    (LONG, 9, 384, 2576),
    (LONG, 0, 1152, 2576),
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("case", range(len(FORMS)))
def test_tiles_in_turn(case, kind, swiglu):
    say("tiles in turn", case, kind, swiglu)
    c = Case(kind, *FORMS[case], swiglu, 200 + case, True)
    got = c.call()
    c.check_all(got)
    np.testing.assert_array_equal(u16(c.call()), u16(got))


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("case", [5, 6, 9])
def test_a_group_of_tiles_does_not_see_the_tiles_before_it(case, kind):
    """NaNs in every other expert's rows, which other tiles of the same workgroups take before and after."""
    counts, spare, depth, n = FORMS[case]
    c = Case(kind, counts, spare, depth, n, False, 300 + case, True)
    plain = u16(c.call())
    ends = np.cumsum(counts)
    keep = np.ones(c.rows, bool)
    for e in range(0, len(counts), 2):
        rows = slice(ends[e] - counts[e], ends[e])
        keep[rows] = False
        if kind == "f8":
            c.a.view(torch.uint8)[rows] = 0x7F
            c.sa[rows] = float("nan")
        else:
            c.a[rows] = float("nan")
    out = c.call()
    np.testing.assert_array_equal(u16(out)[keep], plain[keep])
    assert torch.isnan(out[torch.from_numpy(~keep).to(out.device)]).all()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("depth", [384, 1152, 1040])
def test_int8_tiles_beyond_a_group_of_eight(depth, swiglu):
    say("int8 long groups", depth, swiglu)
    check_product(LONG, 9, depth, 2576, swiglu, depth)
