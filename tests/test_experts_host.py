"""Host-side checks of the experts' entry points (no kernel launched), and
hand-worked pins of their oracle."""
import ctypes
import os
import re
import subprocess
import warnings
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
mod = pytest.importorskip("expert_grouping_dispatch_amd")
P = ctypes.c_void_p
OK_ON_HOST = 3  # MOE_ERR_UNSUPPORTED_DEVICE: the arguments passed every check


def _declared():
    text = open(os.path.join(ROOT, "include", "moe_experts.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(moe_\w+)\s*\(", text, flags=re.M)))


def test_every_declared_symbol_is_exported():
    names = _declared()
    assert names == ["moe_dispatch_i8", "moe_expert_matmul_i8", "moe_layer_few", "moe_layer_few_i64",
                     "moe_layer_few_workspace_bytes", "moe_quantize_i8"]
    out = subprocess.run(["nm", "-D", "--defined-only", mod.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(names) <= exported


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "moe_experts.h"\nint main(void) { return (int)moe_layer_few_workspace_bytes(0, 1, 16); }\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                        os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def _refusals(fn, good, bad):
    """Each (index, value) in turn replaces one good argument; all must be refused with status 1."""
    for at, value in bad:
        args = list(good)
        args[at] = value
        assert fn(*args) == 1, (at, value)


F = P(1 << 20)


def test_dispatch_and_quantize_refusals():
    good = [F, 10, 32, 2, P(1 << 21), P(1 << 22), P(1 << 23), 20, None]
    _refusals(mod.lib.moe_dispatch_i8, good, [(0, None), (0, P(8)), (1, -1), (1, 2 ** 31), (2, 0), (2, 24), (2, -16),
                                              (2, (1 << 20) + 16), (3, 0), (3, 1025), (4, None), (4, P(2)), (5, None),
                                              (5, P(8)), (5, F), (6, None), (6, P(2)), (7, -1)])
    good = [F, 10, 32, None, P(1 << 22), P(1 << 23), None]
    _refusals(mod.lib.moe_quantize_i8, good, [(0, None), (0, P(8)), (1, -1), (1, 2 ** 32 - 1), (2, 0), (2, 40),
                                              (3, P(2)), (4, None), (4, P(8)), (4, F), (4, P((1 << 20) + 32)),
                                              (5, None), (5, P(2))])


MATMUL = [P(1 << 20), P(2 << 20), 10, P(3 << 20), P(4 << 20), 4, P(5 << 20), P(6 << 20), 32, 64, 0, P(7 << 20), None]


def test_matmul_refusals():
    _refusals(mod.lib.moe_expert_matmul_i8, MATMUL,
              [(0, None), (0, P(8)), (1, None), (1, P(2)), (2, -1), (2, 2 ** 32 - 1), (3, None), (3, P(2)), (4, None),
               (4, P(2)), (5, 0), (5, 1025), (6, None), (6, P(8)), (7, None), (7, P(4)), (8, 0), (8, 24),
               (8, (1 << 20) + 16), (9, 0), (9, 24), (9, mod.MATMUL_MAX_DEPTH + 16), (10, 2), (11, None),
               (11, P(8)), (11, MATMUL[0]), (11, MATMUL[6])])


LAYER = [P(1 << 20), 4, 32, 2, P(2 << 20), P(3 << 20), None, 0, 8, P(4 << 20), None, P(5 << 20), None, 48, P(6 << 20),
         P(7 << 20), 1 << 16, None]


def test_layer_refusals():
    for fn in (mod.lib.moe_layer_few, mod.lib.moe_layer_few_i64):
        _refusals(fn, LAYER,
                  [(0, None), (0, P(8)), (1, -1), (1, 1025), (2, 0), (2, 40), (3, 0), (3, 513), (4, None), (4, P(2)),
                   (5, None), (5, P(2)), (6, P(2)), (7, -1), (8, 0), (8, 1025), (9, None), (9, P(8)),
                   (10, P(8 << 20)), (12, P(8 << 20)), (11, None), (11, P(8)), (13, 0), (13, 24), (14, None),
                   (14, P(8)), (14, LAYER[0]), (14, LAYER[11]), (14, LAYER[15]), (15, None), (15, P(128)),
                   (15, LAYER[0]), (15, LAYER[4]), (15, LAYER[9])])
        small = list(LAYER)
        small[16] = mod.moe_layer_few_workspace_bytes(4, 2, 48) - 1
        assert fn(*small) == 2


def test_workspace_size():
    f = mod.moe_layer_few_workspace_bytes
    assert f(0, 1, 16) == 256 and f(4, 2, 48) == 1536 and f(256, 8, 2048) == 256 * 8 * 2048 * 4
    assert f(-1, 1, 16) == f(1, 0, 16) == f(257, 8, 16) == f(1, 2049, 16) == f(1, 1, 24) == f(2 ** 40, 1, 16) == 0
    for n, k, i in ((1, 1, 16), (3, 5, 1040), (256, 8, 7168)):
        assert f(n, k, i) <= 4 * n * k * i + 256 and f(n, k, i) % 256 == 0


def test_outputs_on_inputs_are_refused():
    good = [F, 10, 32, 2, P(1 << 21), P(1 << 22), P(1 << 23), 20, None]
    _refusals(mod.lib.moe_dispatch_i8, good, [(4, good[5]), (4, P((1 << 23) + 76)), (6, F), (6, P((1 << 22) + 636)),
                                              (6, P((1 << 22) - 76)), (5, P((1 << 21) - 624))])
    good = [F, 10, 32, P(1 << 21), P(1 << 22), P(1 << 23), None]
    _refusals(mod.lib.moe_quantize_i8, good, [(5, P((1 << 20) + 636)), (3, P((1 << 22) + 316)), (5, P(1 << 21)),
                                              (5, P((1 << 22) + 316))])
    _refusals(mod.lib.moe_expert_matmul_i8, MATMUL, [(11, MATMUL[i]) for i in (0, 1, 3, 4, 6, 7)] +
              [(3, P((7 << 20) - 16)), (4, P((7 << 20) + 636))])
    layer = list(LAYER)
    layer[6], layer[10], layer[12] = P(10 << 20), P(8 << 20), P(9 << 20)
    for fn in (mod.lib.moe_layer_few, mod.lib.moe_layer_few_i64):
        _refusals(fn, layer, [(out, layer[i]) for out in (14, 15) for i in (0, 4, 5, 6, 9, 10, 11, 12)] +
                  [(6, P((7 << 20) + 1532)), (15, layer[14])])


@pytest.mark.skipif(torch.cuda.is_available(), reason="a HIP device is present: valid arguments would launch")
def test_valid_arguments_reach_the_device_check():
    assert mod.lib.moe_dispatch_i8(F, 10, 32, 2, P(1 << 21), P(1 << 22), P(1 << 23), 20, None) == OK_ON_HOST
    assert mod.lib.moe_dispatch_i8(None, 0, 32, 2, None, None, None, 0, None) == OK_ON_HOST
    assert mod.lib.moe_quantize_i8(F, 10, 32, P(64), P(1 << 22), P(1 << 23), None) == OK_ON_HOST
    assert mod.lib.moe_expert_matmul_i8(*MATMUL) == OK_ON_HOST
    assert mod.lib.moe_layer_few(*LAYER) == OK_ON_HOST
    scaled = list(LAYER)
    scaled[10], scaled[12] = P(8 << 20), P(9 << 20)
    assert mod.lib.moe_layer_few_i64(*scaled) == OK_ON_HOST


@pytest.mark.parametrize("call", ["dispatch", "quantize", "matmul", "layer"])
def test_host_tensors_are_refused(call):
    x, i = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32)
    q, s = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError, match="HIP device"):
        if call == "dispatch":
            mod.moe_dispatch_i8(x, 1, i.view(-1).view(torch.uint32), q, s)
        elif call == "quantize":
            mod.moe_quantize_i8(x, q, s)
        elif call == "matmul":
            mod.moe_expert_matmul_i8(q, s, i.view(-1).view(torch.uint32), i, q, s, x)
        else:
            mod.moe_layer_few(x, i, s, x, x, x, q)


# ---- oracle pins -----------------------------------------------------------------


def _bits(values):
    return (np.asarray(values, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_quantize_pins():
    # largest 127: scale 1, halves go to the even integer
    q, s = oracle.quantize_i8(_bits([[127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -127] * 2]))
    assert s[0] == 1.0 and q[0, :8].tolist() == [127, 0, 2, 2, 0, -2, -2, -127]
    q, s = oracle.quantize_i8(_bits([[254, 3, -5, 1] * 4]))
    assert s[0] == 2.0 and q[0, :4].tolist() == [127, 2, -2, 0]  # 1.5 -> 2, -2.5 -> -2, 0.5 -> 0
    # zeros and values below the floor
    q, s = oracle.quantize_i8(_bits([[0.0] * 16, [2.0 ** -119] * 16]))
    assert s.tolist() == [np.float32(2.0 ** -118 / 127)] * 2 and not q[0].any() and (q[1] == 64).all()


def test_quantize_of_rows_that_are_not_finite():
    """Scale NaN, no cast of a NaN to an integer, the other rows as they are."""
    rows = np.ones((4, 16), np.float32) * 3
    rows[0, 5], rows[2, 0], rows[3, 15] = np.nan, np.inf, -np.inf
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        q, s = oracle.quantize_i8(_bits(rows))
    assert np.isnan(s[[0, 2, 3]]).all() and s[1] == np.float32(3 / 127) and (q[1] == 127).all()


def test_quantize_against_rational_arithmetic():
    g = np.random.default_rng(1)
    x = _bits(g.standard_normal((4, 64)) * np.array([[1e-30], [1.0], [300.0], [1e30]]))
    q, s = oracle.quantize_i8(x)
    v = oracle.bf16_bits_to_f32(x)
    for r in range(4):
        a = max(Fraction(float(t)) for t in np.abs(v[r]))
        assert abs(Fraction(float(s[r])) * 127 / a - 1) <= Fraction(1, 2 ** 23)
        for c in range(64):
            exact = Fraction(float(v[r, c])) * 127 / a
            assert abs(exact - int(q[r, c])) <= Fraction(1, 2) + Fraction(1, 2 ** 16)  # two roundings of 127 at 2^-24
        assert np.abs(q[r]).max() == 127


def test_expert_values_pin():
    v = oracle.expert_values(np.array([[1, -2]], np.int8), np.array([0.5], np.float32),
                             np.array([[3, 4], [-128, 127]], np.int8), np.array([2.0, 0.25], np.float32))
    assert v.tolist() == [[-5.0, -47.75]]
    assert oracle.swiglu(np.array([0.0, 40.0]), np.array([3.0, 3.0])).tolist() == [0.0, 120.0]
    assert abs(oracle.swiglu(np.array([1.0]), np.array([2.0]))[0] - 2 / (1 + np.exp(-1.0))) < 1e-15


def test_layer_pin():
    x = np.array([[20.0, 1.0], [1.0, 1.0]])
    gu = np.array([[[2.0, 0.0], [0.0, 3.0]]])                 # gate = 2 x0, up = 3 x1
    wd = np.array([[[1.0], [-2.0]]])
    out, bound = oracle.layer_few(x, np.array([[0, 0], [-1, 1]]), np.array([[0.5, 1.0], [1.0, 1.0]]), gu, wd)
    assert np.allclose(out, [[180.0, -360.0], [0.0, 0.0]], rtol=1e-12)
    assert (bound[0] > 180 * 2.0 ** -8).all() and (bound[1] <= 2.0 ** -133).all()
