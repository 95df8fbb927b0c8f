"""Host-side checks of the entry points of the experts' products in floating
point (no kernel launched), and hand-worked pins of their oracle."""
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
F8 = torch.float8_e4m3fn


def _declared():
    text = open(os.path.join(ROOT, "include", "moe_experts_float.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(moe_\w+)\s*\(", text, flags=re.M)))


def test_every_declared_symbol_is_exported():
    names = _declared()
    assert names == ["moe_dispatch_f8", "moe_expert_matmul", "moe_expert_matmul_f8", "moe_layer_few_f8",
                     "moe_layer_few_f8_i64", "moe_quantize_f8"]
    out = subprocess.run(["nm", "-D", "--defined-only", mod.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(names) <= exported


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "moe_experts_float.h"\nint main(void) { return MOE_F8_BLOCK == 128 && moe_quantize_f8 ? 0 : 1; }\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wno-address", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                        os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def _refusals(fn, good, bad):
    """Each (index, value) in turn replaces one good argument; all must be refused with status 1."""
    for at, value in bad:
        args = list(good)
        args[at] = value
        assert fn(*args) == 1, (at, value)


F = P(1 << 20)
DISPATCH = [F, 10, 144, 2, P(1 << 21), P(1 << 22), P(1 << 23), 20, None]
QUANTIZE = [F, 10, 144, None, P(1 << 22), P(1 << 23), None]
MATMUL = [P(1 << 20), 10, P(3 << 20), P(4 << 20), 4, P(5 << 20), 32, 144, 0, P(7 << 20), None]
MATMUL_F8 = [P(1 << 20), P(2 << 20), 10, P(3 << 20), P(4 << 20), 4, P(5 << 20), P(6 << 20), 144, 144, 1, P(7 << 20), None]


def test_dispatch_and_quantize_refusals():
    _refusals(mod.lib.moe_dispatch_f8, DISPATCH,
              [(0, None), (0, P(8)), (1, -1), (1, 2 ** 31), (2, 0), (2, 24), (2, -16), (2, (1 << 20) + 16), (3, 0),
               (3, 1025), (4, None), (4, P(2)), (5, None), (5, P(8)), (5, F), (6, None), (6, P(2)), (7, -1)])
    _refusals(mod.lib.moe_quantize_f8, QUANTIZE,
              [(0, None), (0, P(8)), (1, -1), (1, 2 ** 32 - 1), (2, 0), (2, 40), (3, P(2)), (4, None), (4, P(8)),
               (4, F), (5, None), (5, P(2))])


def test_matmul_refusals():
    _refusals(mod.lib.moe_expert_matmul, MATMUL,
              [(0, None), (0, P(8)), (1, -1), (1, 2 ** 32 - 1), (2, None), (2, P(2)), (3, None), (3, P(2)), (4, 0),
               (4, 1025), (5, None), (5, P(8)), (6, 0), (6, 24), (6, (1 << 20) + 16), (7, 0), (7, 24),
               (7, mod.MATMUL_MAX_DEPTH + 16), (8, 2), (9, None), (9, P(8))])
    _refusals(mod.lib.moe_expert_matmul_f8, MATMUL_F8,
              [(0, None), (0, P(8)), (1, None), (1, P(2)), (2, -1), (2, 2 ** 32 - 1), (3, None), (3, P(2)), (4, None),
               (4, P(2)), (5, 0), (5, 1025), (6, None), (6, P(8)), (7, None), (7, P(2)), (8, 0), (8, 24),
               (8, (1 << 20) + 16), (9, 0), (9, 24), (9, mod.MATMUL_MAX_DEPTH + 16), (10, 2), (11, None), (11, P(8))])


def test_outputs_on_inputs_are_refused():
    # two blocks a row: 8 bytes of scales; the last bytes of each buffer count
    _refusals(mod.lib.moe_dispatch_f8, DISPATCH, [(4, DISPATCH[5]), (4, P((1 << 23) + 156)), (6, F),
                                                  (6, P((1 << 22) + 20 * 144 - 4)), (6, P((1 << 22) - 156)),
                                                  (5, P((1 << 20) + 10 * 288 - 16))])
    _refusals(mod.lib.moe_quantize_f8, QUANTIZE, [(5, P((1 << 20) + 10 * 288 - 4)), (3, P((1 << 22) + 1436)),
                                                  (3, P((1 << 23) + 76)), (5, P((1 << 22) + 1436))])
    _refusals(mod.lib.moe_expert_matmul, MATMUL, [(9, MATMUL[i]) for i in (0, 2, 3, 5)] +
              [(2, P((7 << 20) - 16)), (3, P((7 << 20) + 636)), (0, P((7 << 20) - 2864)), (5, P((7 << 20) - 36848))])
    # 2 halves of 2 x 2 blocks for each of 4 experts: 128 bytes of scales
    _refusals(mod.lib.moe_expert_matmul_f8, MATMUL_F8, [(11, MATMUL_F8[i]) for i in (0, 1, 3, 4, 6, 7)] +
              [(1, P((7 << 20) - 76)), (7, P((7 << 20) - 124)), (6, P((7 << 20) - 4 * 288 * 144 + 16))])


LAYER = [P(1 << 20), 4, 144, 2, P(2 << 20), P(3 << 20), P(10 << 20), 0, 8, P(4 << 20), P(8 << 20), P(5 << 20),
         P(9 << 20), 48, P(6 << 20), P(7 << 20), 1 << 16, None]
LAYERS = (mod.lib.moe_layer_few_f8, mod.lib.moe_layer_few_f8_i64)


@pytest.mark.parametrize("fn", LAYERS)
def test_layer_refusals(fn):
    _refusals(fn, LAYER,
              [(0, None), (0, P(8)), (1, -1), (1, 1025), (2, 0), (2, 40), (2, (1 << 17) + 16), (3, 0), (3, 513),
               (4, None), (4, P(2)), (5, None), (5, P(2)), (6, P(2)), (7, -1), (8, 0), (8, 1025), (9, None), (9, P(8)),
               (10, None), (10, P(2)), (11, None), (11, P(8)), (12, None), (12, P(2)), (13, 0), (13, 24),
               (13, (1 << 17) + 16), (14, None), (14, P(8)), (15, None), (15, P(128))])
    # 2 blocks of hidden, 1 of inter: 8 experts' scales are 128 and 64 bytes
    _refusals(fn, LAYER, [(out, LAYER[i]) for out in (14, 15) for i in (0, 4, 5, 6, 9, 10, 11, 12)] +
              [(10, P((6 << 20) - 124)), (12, P((6 << 20) - 60)), (6, P((7 << 20) + 1532)), (15, LAYER[14])])
    small = list(LAYER)
    small[16] = mod.moe_layer_few_workspace_bytes(4, 2, 48) - 1
    assert fn(*small) == 2
    both = list(LAYER)
    both[10] = both[12] = None  # no scales: not bf16 weights, refused
    assert fn(*both) == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="a HIP device is present: valid arguments would launch")
def test_valid_arguments_reach_the_device_check():
    assert mod.lib.moe_dispatch_f8(*DISPATCH) == OK_ON_HOST
    assert mod.lib.moe_dispatch_f8(None, 0, 32, 2, None, None, None, 0, None) == OK_ON_HOST
    assert mod.lib.moe_quantize_f8(*QUANTIZE) == OK_ON_HOST
    assert mod.lib.moe_quantize_f8(F, 10, 32, P(64), P(1 << 22), P(1 << 23), None) == OK_ON_HOST
    assert mod.lib.moe_expert_matmul(*MATMUL) == OK_ON_HOST
    assert mod.lib.moe_expert_matmul_f8(*MATMUL_F8) == OK_ON_HOST
    for fn in LAYERS:
        assert fn(*LAYER) == OK_ON_HOST
        beside = list(LAYER)
        beside[10], beside[12] = P((6 << 20) - 128), P((6 << 20) + 4 * 288)
        assert fn(*beside) == OK_ON_HOST
    beside = list(MATMUL_F8)  # buffers that touch and do not overlap
    beside[1], beside[7] = P((7 << 20) - 80), P((7 << 20) + 10 * 288)
    assert mod.lib.moe_expert_matmul_f8(*beside) == OK_ON_HOST


@pytest.mark.parametrize("call", ["dispatch", "quantize", "matmul", "matmul_f8", "layer"])
def test_host_tensors_are_refused(call):
    x, i = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32)
    q, s = torch.zeros(2, 32).to(F8), torch.zeros(2, 1)
    with pytest.raises(ValueError, match="HIP device"):
        if call == "dispatch":
            mod.moe_dispatch_f8(x, 1, i.view(-1).view(torch.uint32), q, s)
        elif call == "quantize":
            mod.moe_quantize_f8(x, q, s)
        elif call == "matmul":
            mod.moe_expert_matmul(x, i.view(-1).view(torch.uint32), i, x, x)
        elif call == "layer":
            mod.moe_layer_few(x, i, s, q, q, x, q, gate_up_scales=s, down_scales=s)
        else:
            mod.moe_expert_matmul_f8(q, s, i.view(-1).view(torch.uint32), i, q, s, x)


# ---- oracle pins -----------------------------------------------------------------


def _bits(values):
    return (np.asarray(values, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(F8).double().numpy()
    np.testing.assert_array_equal(oracle.e4m3_values(), want)


def test_e4m3_codes():
    """Every value, every midpoint and its neighbours, against torch's rounding."""
    v = oracle.e4m3_values()[:127]
    mid = (v[1:] + v[:-1]) / 2
    t = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64), [448.00003, 0.0]])
    t = np.concatenate([t, -t])
    want = torch.from_numpy(t).float().to(F8).view(torch.uint8).numpy()
    np.testing.assert_array_equal(oracle.e4m3_codes(t), want)
    # 0x38 is 1, a step is 1/8: 1 + 1/16 is a tie and goes to the even code, 1 + 3/16 to the next even one
    assert oracle.e4m3_codes(np.array([1.0, 1.0625, 1.1875, -1.0625])).tolist() == [0x38, 0x38, 0x3A, 0xB8]


def test_quantize_f8_pins():
    row = [448, 1.0625, -17, 2.0 ** -9, 2.0 ** -10, -0.0] + [0] * 122  # scale 1
    second = [896, 3, -34, 0]                                           # a short block, scale 2
    q, s = oracle.quantize_f8(_bits([row + second + [0] * 12]))
    assert s.tolist() == [[1.0, 2.0]]
    assert q[0, :6].tolist() == [0x7E, 0x38, 0xD8, 0x01, 0x00, 0x80]    # -17 is a tie of -16 and -18
    assert q[0, 128:132].tolist() == [0x7E, 0x3C, 0xD8, 0x00]
    q, s = oracle.quantize_f8(_bits([[0.0] * 16, [2.0 ** -117] * 16]))
    assert s[:, 0].tolist() == [np.float32(2.0 ** -116 / 448)] * 2 and not q[0].any()
    assert (oracle.e4m3_values()[q[1]] == 224).all()


def test_quantize_f8_of_blocks_that_are_not_finite():
    rows = np.full((3, 272), 3, np.float32)
    rows[0, 5], rows[1, 128], rows[2, 271] = np.nan, np.inf, -np.inf
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        q, s = oracle.quantize_f8(_bits(rows))
    assert np.isnan(s).tolist() == [[True, False, False], [False, True, False], [False, False, True]]
    assert (s[~np.isnan(s)] == np.float32(3 / 448)).all() and (q[0, 128:] == 0x7E).all()


def test_quantize_f8_against_rational_arithmetic():
    g = np.random.default_rng(1)
    x = _bits(g.standard_normal((4, 144)) * np.array([[1e-30], [1.0], [300.0], [1e30]]))
    q, s = oracle.quantize_f8(x)
    v, values = oracle.bf16_bits_to_f32(x), oracle.e4m3_values()
    for r in range(4):
        for b in range(2):
            block = v[r, 128 * b:128 * (b + 1)]
            a = max(Fraction(float(t)) for t in np.abs(block))
            assert abs(Fraction(float(s[r, b])) * 448 / a - 1) <= Fraction(1, 2 ** 23)
            for c in range(block.size):
                exact = Fraction(float(block[c])) * 448 / a
                got = Fraction(float(values[q[r, 128 * b + c]]))
                # half a step: 2^-4 of the value, 2^-10 among the subnormals; two roundings at 2^-24
                assert abs(exact - got) <= max(abs(exact) / 16, Fraction(1, 2 ** 10)) * (1 + Fraction(1, 2 ** 20))


def test_block_weights_and_products_pin():
    w = np.ones((2 * 130, 129))
    s = np.arange(1.0, 9.0).reshape(4, 2)
    v = oracle.block_weights(w, s, halves=2)
    assert v[0, 0] == 1 and v[0, 128] == 2 and v[127, 0] == 1 and v[128, 0] == 3 and v[129, 128] == 4
    assert v[130, 0] == 5 and v[257, 128] == 6 and v[258, 0] == 7 and v[259, 128] == 8
    out, bound = oracle.products(np.array([[1.0, -2.0]]), np.array([[3.0, 4.0], [-128.0, 127.0]]), False)
    assert out.tolist() == [[-5.0, -382.0]] and (bound >= np.abs(out) / 256).all() and (bound < np.abs(out) / 250).all()
    # e4m3: seven products of an eight may lose 2^-13 of the largest each
    a8, w8 = np.array([[256.0, -256.0] + [1.0] * 6]), np.array([[256.0, 256.0] + [1.0] * 6])
    plain, cut = (oracle.products(a8, w8, False, f8)[1][0, 0] for f8 in (False, True))
    assert oracle.products(a8, w8, False, True)[0][0, 0] == 6 and abs(cut - plain - 56 * (1 + 2.0 ** -8)) < 1e-3
    out, bound = oracle.products(np.array([[40.0]]), np.array([[1.0], [0.5]]), True)
    assert abs(out[0, 0] - 800) < 1e-9 and 800 / 256 <= bound[0, 0] < 3.2
