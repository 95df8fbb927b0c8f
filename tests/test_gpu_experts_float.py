"""The experts' products in floating point on the GPU.

Dispatch and quantisation are bit-exact by their definitions.  The products are
compared bit for bit on whole numbers and powers of two, where every partial
sum is exact in fp32 whatever its order, and on normal values with the oracle's
bound.  With SwiGLU the whole numbers' gate and up are exact; half a bf16 step
(2^-8) and the fp32 evaluation of silu(gate) * up count, (104 + 8) 2^-24 < 2^-17
relative, as |gate| < 104 wherever silu(gate) is not below every bf16 value."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_common import bf16_from_bits, gpu_available, u16
from tests.test_gpu_experts import SILU, TINY, _csr, bf16_rows, dev, f64

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

mod = pytest.importorskip("expert_grouping_dispatch_amd") if gpu_available() else None
DEV = "cuda"
F8 = torch.float8_e4m3fn


def say(*a):
    print("[experts float]", *a, flush=True)


def blocks(n):
    return -(-n // 128)


def codes(q):
    return q.view(torch.uint8).cpu().numpy()


def u32_of(a):
    return dev(np.asarray(a, np.uint32).view(np.int32)).view(torch.uint32)


# ---- rows in e4m3 -------------------------------------------------------------------


def _f8_rows(g, n, h):
    """Rows as for int8, with blocks of very different size beside each other."""
    xb = bf16_rows(g, n, h)
    for r in range(0, n, 5):
        v = g.standard_normal(h) * np.exp2(g.integers(-60, 60, blocks(h)))[np.arange(h) // 128]
        xb[r] = oracle.f32_to_bf16_rne(v.astype(np.float32))
    return xb


@pytest.mark.parametrize("n, h, count", [(1, 16, None), (9, 48, 5), (30, 1040, 0), (30, 7168, 29), (8, 8208, None),
                                         (8, 16400, 2 ** 32 - 1), (9, 32784, 7), (2100, 272, 2077), (40, 128, 33),
                                         (17, 1024, None), (5, 2064, 4)])
def test_quantize(n, h, count):
    say("quantize", n, h, count)
    xb = _f8_rows(np.random.default_rng(n * h), n, h)
    q = torch.full((n, h), 77, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.full((n, blocks(h)), -3.0, device=DEV)
    mod.moe_quantize_f8(bf16_from_bits(xb, DEV), q, s, None if count is None else u32_of([count]))
    real = n if count is None else min(n, count)
    wq, ws = oracle.quantize_f8(xb)
    np.testing.assert_array_equal(codes(q)[:real], wq[:real])
    np.testing.assert_array_equal(s.cpu().numpy()[:real], ws[:real])
    assert (codes(q)[real:] == 77).all() and (s[real:] == -3.0).all()


def test_quantize_every_bf16_value():
    """All finite bf16 values, each beside a largest value that makes the block's scale 1, 2^-8 or 2^20."""
    every = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    every = every[(every & 0x7F80) != 0x7F80]
    for largest in (448.0, 1.75, 448.0 * 2 ** 20):
        top = oracle.f32_to_bf16_rne(np.float32([largest]))[0]
        xb = every[(oracle.bf16_bits_to_f32(every) <= largest) & (oracle.bf16_bits_to_f32(every) >= -largest)]
        xb = np.concatenate([xb, np.zeros(-xb.size % 127, np.uint16)]).reshape(-1, 127)
        xb = np.concatenate([np.full((xb.shape[0], 1), top, np.uint16), xb], axis=1)
        q, s = mod.alloc_quantized_f8(*xb.shape, DEV)
        mod.moe_quantize_f8(bf16_from_bits(xb, DEV), q, s)
        wq, ws = oracle.quantize_f8(xb)
        np.testing.assert_array_equal(codes(q), wq)
        np.testing.assert_array_equal(s.cpu().numpy(), ws)


def test_quantize_streams_past_the_caches():
    """More than the Infinity Cache holds: the form with non-temporal loads and stores, ragged rows."""
    n, h = 6000, 15120
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((n, h), generator=g, device=DEV).to(torch.bfloat16)
    q, s = mod.alloc_quantized_f8(n, h, DEV)
    mod.moe_quantize_f8(x, q, s)
    v = torch.nn.functional.pad(x.float(), (0, -h % 128)).view(n, -1, 128)
    a = v.abs().amax(2).double()
    assert torch.equal(s, (a / 448).float())
    want = (v * (448 / a).float()[:, :, None]).to(F8).view(n, -1)[:, :h]
    assert torch.equal(q.view(torch.uint8), want.contiguous().view(torch.uint8))


def test_quantize_blocks_with_infinities_and_nans_have_scale_nan():
    g = np.random.default_rng(5)
    xb = oracle.f32_to_bf16_rne(g.standard_normal((6, 1040)).astype(np.float32))
    xb[1, 1039], xb[3, 0], xb[4, 500] = 0x7F80, 0x7FC0, 0xFF80
    q, s = mod.alloc_quantized_f8(6, 1040, DEV)
    mod.moe_quantize_f8(bf16_from_bits(xb, DEV), q, s)
    wq, ws = oracle.quantize_f8(xb)
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    assert np.isnan(ws).sum() == 3
    fine = ~np.isnan(ws)[:, np.arange(1040) // 128]
    np.testing.assert_array_equal(codes(q)[fine], wq[fine])


@pytest.mark.parametrize("n, k, e, h, spare", [(1, 1, 4, 16, 0), (33, 2, 8, 256, 0), (50, 8, 64, 1040, -30),
                                               (40, 9, 32, 272, 0), (7, 3, 5, 32784, 0), (13, 20, 6, 7168, 4),
                                               (300, 5, 12, 2064, 0)])
def test_dispatch(n, k, e, h, spare):
    """Padding rows hold NaN and are not read; with a short output the positions behind it are skipped."""
    say("dispatch", n, k, e, h)
    g = np.random.default_rng(n + k)
    ids = g.integers(-1, e + 1, (n, k)).astype(np.int32)   # repeats, -1 and an id past the end
    ids[n - n // 4:] = -1
    xb = _f8_rows(g, n, h)
    xb[(ids < 0).all(1) | (ids >= e).all(1)] = 0x7FC0
    ref = oracle.create_indices(ids, e)
    v, rows = ref["n_routed"], n * k + spare
    q = torch.full((rows, h), 77, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.full((rows, blocks(h)), -3.0, device=DEV)
    mod.moe_dispatch_f8(bf16_from_bits(xb, DEV), k, u32_of(ref["restore_token_order"]), q, s)
    m = min(v, rows)
    wq, ws = oracle.dispatch_f8(xb, ref["token_expert_order"], k, v)
    np.testing.assert_array_equal(codes(q)[:m], wq[:m])
    np.testing.assert_array_equal(s.cpu().numpy()[:m], ws[:m])
    assert (codes(q)[m:] == 77).all() and (s[m:] == -3.0).all()


def test_rows_beyond_4_gib():
    """Byte offsets pass 32 bits in the payload: of the last rows in order, and of the places that slots map to."""
    h = 8192
    n = 2 ** 32 // h + 37
    say("rows beyond 4 GiB", n, h)
    xb = _f8_rows(np.random.default_rng(41), 40, h)
    wq, ws = oracle.quantize_f8(xb)
    x = torch.zeros((n, h), dtype=torch.bfloat16, device=DEV)
    x[n - 40:] = bf16_from_bits(xb, DEV)
    q, s = mod.alloc_quantized_f8(n, h, DEV)
    mod.moe_quantize_f8(x, q, s)
    np.testing.assert_array_equal(codes(q[n - 40:]), wq)
    np.testing.assert_array_equal(s[n - 40:].cpu().numpy(), ws)
    assert not codes(q[:50]).any() and (s[:50] == 2.0 ** -116 / 448).all()
    q.view(torch.uint8).fill_(77), s.fill_(-3.0)
    places = np.stack([np.arange(40), n - 1 - np.arange(40)], 1)  # each row at both ends
    mod.moe_dispatch_f8(x[n - 40:], 2, u32_of(places.reshape(-1)), q, s)
    for at in (slice(0, 40), slice(n - 40, n)):
        order = slice(None) if at.start == 0 else slice(None, None, -1)
        np.testing.assert_array_equal(codes(q[at]), wq[order])
        np.testing.assert_array_equal(s[at].cpu().numpy(), ws[order])
    assert (codes(q[40:90]) == 77).all() and (codes(q[n - 90:n - 40]) == 77).all()


# ---- grouped products ----------------------------------------------------------------


class Case:
    """Operands of a grouped product on the GPU and what they stand for, in 64 bits."""

    def __init__(self, kind, counts, spare, depth, n, swiglu, seed, whole):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.kind, self.counts, self.n, self.depth, self.swiglu = kind, counts, n, depth, swiglu
        halves, e, rows = 2 if swiglu else 1, len(counts), sum(counts) + spare
        self.starts, self.ids = _csr(counts)

        def ints(most, *shape):
            return torch.randint(-most, most + 1, shape, generator=g, device=DEV, dtype=torch.int8)

        def normal(*shape):
            return torch.randn(shape, generator=g, device=DEV)

        f8 = kind == "f8"
        if whole:  # |a| |w| < 400, scales of at most 2: below 2^24 steps of the least one for any depth up to 10000
            a, w = ints(15 if f8 else 127, rows, depth), ints(3, e, halves * n, depth)
            size = 2.0 ** -6  # gates of a few units
        else:
            a, w, size = normal(rows, depth), normal(e, halves * n, depth), depth ** -0.5
        if f8:
            per_a, per_w = (rows, blocks(depth)), (e, halves * blocks(n), blocks(depth))
            if whole:
                self.sa, self.sw = torch.exp2(ints(1, *per_a).float()), torch.exp2(ints(1, *per_w).float()) * size
                self.a, self.w = a.float().to(F8), w.float().to(F8)
            else:
                self.sa = (0.5 + torch.rand(per_a, generator=g, device=DEV)) / 165
                self.sw = (0.5 + torch.rand(per_w, generator=g, device=DEV)) * size / 105
                self.a, self.w = (a * 165).clamp(-448, 448).to(F8), (w * 105).clamp(-448, 448).to(F8)
        else:
            self.sa = self.sw = None
            self.a, self.w = a.to(torch.bfloat16), (w * size).to(torch.bfloat16)
        self.rows = rows
        v = sum(counts)  # nothing may come of what lies behind the last group
        if f8:
            self.a.view(torch.uint8)[v:] = 0x7F
            self.sa[v:] = float("nan")
        else:
            self.a[v:] = float("nan")

    def values(self, lo, hi, e):
        """Rows lo .. hi and the weights of expert e in 64 bits."""
        a, w = self.a[lo:hi].double(), self.w[e].double()
        if self.kind == "f8":
            k = torch.arange(self.depth, device=DEV) // 128
            a *= self.sa[lo:hi].double()[:, k]
            half = self.sw[e].double().view(2 if self.swiglu else 1, blocks(self.n), -1)
            w *= half[:, torch.arange(self.n, device=DEV) // 128][:, :, k].reshape(w.shape)
        return a, w

    def call(self, out=None, starts=None, ids=None):
        if out is None:
            out = torch.full((self.rows, self.n), 7.0, dtype=torch.bfloat16, device=DEV)
        starts, ids = u32_of(self.starts if starts is None else starts), dev(self.ids if ids is None else ids)
        flags = mod.MATMUL_SWIGLU if self.swiglu else 0
        if self.kind == "f8":
            mod.moe_expert_matmul_f8(self.a, self.sa, starts, ids, self.w, self.sw, out, flags=flags)
        else:
            mod.moe_expert_matmul(self.a, starts, ids, self.w, out, flags=flags)
        return out

    def check_whole(self, got, lo, hi, e, message=""):
        a, w = self.values(lo, hi, e)
        y = torch.mm(a, w.t())
        assert torch.mm(a.abs(), w.abs().t()).max() < 2.0 ** 24 * 2.0 ** -8
        if self.swiglu:
            gate, up = y[:, :self.n], y[:, self.n:]
            want = gate * torch.special.expit(gate) * up
            # exp(-gate) passes fp32's largest number, and silu(gate) becomes -0, from gate < -128 ln 2 = -88.72 on,
            # where |gate| exp(gate) falls: |silu(gate)| < 88.73 * 2^-128 < 2^-121.
            bad = ~((got.double() - want).abs() <= SILU * want.abs() + TINY + 2.0 ** -121 * up.abs())
            assert not bad.any(), (message, e, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())
        else:
            np.testing.assert_array_equal(u16(got), u16(y.float().to(torch.bfloat16)), err_msg=f"{message} expert {e}")

    def check_all(self, out):
        v, at = sum(self.counts), 0
        assert (out[v:] == 7.0).all()
        for e, c in enumerate(self.counts):
            if c:
                self.check_whole(out[at:at + c], at, at + c, e, f"{c} rows,")
            at += c


MIXED = [300, 100, 256, 70, 129, 513, 66, 200]  # tiles of 65..128 and of 129..256 rows beside each other
FORMS = [
    # counts per expert, spare rows, depth, weight rows per expert (doubled with SwiGLU)
    ([1], 0, 16, 16),
    ([0, 0, 0], 5, 64, 32),
    ([3, 0, 16, 1], 2, 48, 48),
    ([17, 33, 0, 64, 15], 7, 144, 80),
    ([65], 0, 128, 16),
    ([65, 2, 128, 0, 70], 30, 272, 272),
    ([255, 256, 257, 1], 3, 400, 144),
    ([700, 0, 20], 0, 1040, 528),
    ([0] * 40 + [90, 3] + [0] * 20, 9, 656, 1040),
    ([5] * 300, 11, 80, 64),
    ([70] * 24, 1, 2064, 320),
    ([2, 33, 64, 17, 1, 32, 48, 0] * 26, 5, 272, 528),   # strips of up to 32 and up to 64 rows
    ([64, 63, 32, 31] * 20, 5, 1936, 1040),
    ([40] * 130, 0, 4096, 400),
    ([1, 90, 16, 31] * 40, 0, 128, 1040),                # strips and tiles
    (MIXED, 11, 896, 912),
    (MIXED, 11, 912, 784),
    ([1] * 1024, 0, 64, 48),
    ([100] * 9, 0, 64, 4112),                            # one step, many tiles for each workgroup
    ([100, 300] * 40, 3, 192, 1040),
    ([9, 60], 0, 8192, 16),                              # few rows, long sums
    ([500], 0, 8208, 272),
    ([4000], 0, 256, 256),
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("case", range(len(FORMS)))
def test_matmul_on_whole_numbers(case, kind, swiglu):
    say("matmul whole", case, kind, swiglu)
    c = Case(kind, *FORMS[case], swiglu, case, True)
    c.check_all(c.call())


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("case", [3, 5, 6, 7, 11, 12, 16, 20])
def test_matmul_against_the_bound(case, kind, swiglu):
    say("matmul", case, kind, swiglu)
    c = Case(kind, *FORMS[case], swiglu, 50 + case, False)
    out, at = c.call(), 0
    for e, n in enumerate(c.counts):
        if n:
            want, bound = oracle.products(*(f64(t) for t in c.values(at, at + n, e)), swiglu, kind == "f8")
            bad = ~(np.abs(f64(out[at:at + n]) - want) <= bound)
            assert not bad.any(), (e, np.argwhere(bad)[:4], f64(out[at:at + n])[bad][:4], want[bad][:4], bound[bad][:4])
        at += n


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("counts, n", [([8], 16), ([8, 40] * 130, 16), ([80, 200], 272)])
def test_matmul_small_products_beside_large_ones(kind, counts, n):
    """Pairs of +-2^16 that cancel, with products of 2^-18 to 2^12 in the same eight, in the same sixteen and further
    off: what the sums may lose is bounded, in bf16 by fp32 alone."""
    depth = 272
    c = Case(kind, counts, 0, depth, n, False, 12, True)
    g = np.random.default_rng(13)
    a = np.exp2(g.integers(-9, 7, (c.rows, depth)).astype(np.float64)) * g.choice([-1, 1], (c.rows, depth))
    w = np.exp2(g.integers(-9, 7, (len(counts), n, depth)).astype(np.float64))
    for at in (0, 7, 17, 40, 41, 130, 200, 270):
        a[:, at] = w[:, :, at] = 256
        other = at + 1 if at % 2 == 0 else at - 1 if at != 41 else 43
        a[:, other], w[:, :, other] = 256, -256
    c.a, c.w = dev(a.astype(np.float32)).to(c.a.dtype), dev(w.astype(np.float32)).to(c.w.dtype)
    if kind == "f8":
        c.sa.fill_(1.0)
        c.sw.fill_(1.0)
    out, at = c.call(), 0
    for e, m in enumerate(counts):
        want, bound = oracle.products(a[at:at + m], w[e], False, kind == "f8")
        bad = ~(np.abs(f64(out[at:at + m]) - want) <= bound)
        assert not bad.any(), (e, np.argwhere(bad)[:4], f64(out[at:at + m])[bad][:4], want[bad][:4], bound[bad][:4])
        at += m


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("counts, n", [([20, 30], 80), ([20, 30] * 40, 1040), ([200, 90], 80)])
def test_matmul_rows_and_experts_that_are_not_finite_stay_alone(kind, counts, n):
    """Rows of NaN, and the weights of an expert without rows, beside rows that end inside a step."""
    depth = 144
    c = Case(kind, counts + [0], 0, depth, n, False, 3, True)
    plain = c.call()
    c.check_all(plain)
    bad = [7, counts[0] + 3]
    if kind == "f8":
        c.a.view(torch.uint8)[bad[0]] = 0x7F
        c.sa[bad[1], 1] = float("inf")
        c.w.view(torch.uint8)[len(counts)] = 0x7F
        c.sw[len(counts)] = float("nan")
    else:
        c.a[bad[0]], c.a[bad[1]], c.w[len(counts)] = float("nan"), float("inf"), float("nan")
    out = c.call()
    keep = np.ones(sum(counts), bool)
    keep[bad] = False
    assert torch.isnan(out[bad[0]]).all() and not torch.isfinite(out[bad[1]]).any()
    np.testing.assert_array_equal(u16(out)[keep], u16(plain)[keep])


def _moved(t, values):
    """A copy of t that begins `values` elements into its memory, between NaNs (or 7s) that nothing may come of."""
    fill = 0x7F if t.dtype == F8 else float("nan") if t.is_floating_point() else 7
    room = torch.empty(t.numel() + 2 * values, dtype=t.dtype, device=DEV)
    (room.view(torch.uint8) if t.dtype == F8 else room).fill_(fill)
    room[values:values + t.numel()] = t.reshape(-1)
    return room[values:values + t.numel()].view(t.shape)


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("case", [2, 5, 11, 15, 21])
def test_matmul_with_the_least_alignment(case, kind, swiglu):
    """Operands at 16 bytes, scales at 4: the same bits."""
    c = Case(kind, *FORMS[case], swiglu, case, True)
    want = u16(c.call())
    c.a, c.w = (_moved(t, 16 // t.element_size()) for t in (c.a, c.w))
    for values in (1, 3):
        if kind == "f8":
            c.sa, c.sw = _moved(c.sa, values), _moved(c.sw, values)
        out = _moved(torch.full((c.rows, c.n), 7.0, dtype=torch.bfloat16, device=DEV), 8)
        np.testing.assert_array_equal(u16(c.call(out=out)), want)


@pytest.mark.parametrize("counts, depth", [([20], 16), ([200, 90], 112), ([200, 90], 128), ([20, 30] * 40, 128),
                                           ([300, 70], 640)])
def test_matmul_f8_scales_that_are_not_finite(counts, depth):
    """An infinite or NaN scale of a row, or of a block of an expert's weights, is in all of that row's or of those
    channels' outputs, and in no other."""
    n = 272
    c = Case("f8", counts, 0, depth, n, False, 6, True)
    plain = c.call()
    rows, last = [3, counts[0] - 1], blocks(depth) - 1
    c.sa[rows[0], 0], c.sa[rows[1], last] = float("inf"), float("nan")
    c.sw[-1, 0, last], c.sw[-1, 2, 0] = float("-inf"), float("nan")
    out = c.call()
    hit = torch.zeros((c.rows, n), dtype=torch.bool, device=DEV)
    hit[rows] = True
    hit[c.rows - counts[-1]:, :128] = True
    hit[c.rows - counts[-1]:, 256:] = True
    assert not torch.isfinite(out[hit]).any()
    np.testing.assert_array_equal(u16(out)[~hit.cpu().numpy()], u16(plain)[~hit.cpu().numpy()])


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_matmul_bad_data_stays_inside_the_buffers(kind, swiglu):
    """An active expert with an id out of range is skipped; starts behind the buffer's end count as its end, and
    starts that fall make an empty group."""
    c = Case(kind, [20, 100, 10, 300, 5], 0, 64, 32, swiglu, 4, True)
    starts, ids = c.starts.copy(), c.ids.copy()
    starts[5], ids[1], ids[2] = 5000, 77, -5
    out = c.call(starts=starts, ids=ids)
    assert (out[20:130] == 7.0).all()
    c.check_whole(out[:20], 0, 20, 0)
    c.check_whole(out[130:430], 130, 430, 3)
    c.check_whole(out[430:], 430, 435, 4)
    starts[3] = 2  # the third group is empty, the fourth lies on the first two: rows 2 to 119 have two experts
    out = c.call(starts=starts, ids=c.ids)
    c.check_whole(out[:2], 0, 2, 0)
    c.check_whole(out[120:430], 120, 430, 3)
    c.check_whole(out[430:], 430, 435, 4)


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("rows", [3, 60, 300])
def test_matmul_with_weights_beyond_4_gib(kind, rows):
    """Byte offsets of the last expert's weights pass 32 bits."""
    e, depth, n = (70, 8192, 8192) if kind == "f8" else (40, 8192, 8192)
    say("matmul large weights", kind, rows)
    one = Case(kind, [rows, rows], 0, depth, n, False, 5, True)
    w = torch.zeros((e, n, depth), dtype=one.w.dtype, device=DEV)
    w[0], w[e - 1] = one.w[0], one.w[1]
    out = torch.full((2 * rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
    starts, ids = _csr([rows] + [0] * (e - 2) + [rows])
    if kind == "f8":
        sw = torch.ones((e, *one.sw.shape[1:]), device=DEV)
        sw[0], sw[e - 1] = one.sw[0], one.sw[1]
        mod.moe_expert_matmul_f8(one.a, one.sa, u32_of(starts), dev(ids), w, sw, out)
    else:
        mod.moe_expert_matmul(one.a, u32_of(starts), dev(ids), w, out)
    one.check_whole(out[:rows], 0, rows, 0)
    one.check_whole(out[rows:], rows, 2 * rows, 1)


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("last", [10, 200])
def test_matmul_with_rows_beyond_4_gib(kind, last):
    """Byte offsets of the last group's rows pass 32 bits in the operand and, but for e4m3, in the output; the rows
    before it belong to an id out of range and are not read."""
    depth, n = 8192, 8192 if kind == "bf16" else 4112
    before = 2 ** 32 // (depth * (2 if kind == "bf16" else 1)) + 100
    say("matmul large rows", kind, last)
    c = Case(kind, [last], 0, depth, n, False, 6, True)
    a = torch.zeros((before + last, depth), dtype=c.a.dtype, device=DEV)
    a[before:] = c.a
    out = torch.full((before + last, n), 7.0, dtype=torch.bfloat16, device=DEV)
    starts, ids = u32_of([0, before, before + last]), dev(np.array([-1, 0], np.int32))
    w = torch.cat((c.w, torch.zeros_like(c.w)))
    if kind == "f8":
        sa = torch.full((before + last, blocks(depth)), float("nan"), device=DEV)
        sa[before:] = c.sa
        mod.moe_expert_matmul_f8(a, sa, starts, ids, w, torch.cat((c.sw, c.sw)), out)
    else:
        mod.moe_expert_matmul(a, starts, ids, w, out)
    c.check_whole(out[before:], 0, last, 0)
    assert (out[:100] == 7.0).all() and (out[before - 100:before] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "f8"])
def test_matmul_longest_rows(kind):
    """The largest depth, few rows and a tile: ones and powers of two, sums of 131056 exactly."""
    depth = mod.MATMUL_MAX_DEPTH
    for counts in ([40], [130]):
        say("matmul longest", kind, counts)
        c = Case(kind, counts, 0, depth, 16, False, 7, True)
        c.a, c.w = torch.ones_like(c.a.float()).to(c.a.dtype), torch.ones_like(c.w.float()).to(c.w.dtype)
        c.w[0, 1] = torch.full((depth,), 0.5).to(c.w.dtype)
        if kind == "f8":
            c.sa.fill_(2.0)
            c.sw.fill_(0.25)
        out = c.call()
        want = depth * (0.5 if kind == "f8" else 1.0)
        row = torch.full((16,), want, device=DEV)
        row[1] /= 2
        np.testing.assert_array_equal(u16(out), u16(row.to(torch.bfloat16).expand_as(out)))


@pytest.mark.parametrize("kind", ["bf16", "f8"])
def test_matmul_repeats_bit_for_bit_and_two_streams_do_not_meet(kind):
    cases = [Case(kind, MIXED, 0, 912, 784, True, 8, False), Case(kind, [20, 33, 5] * 50, 0, 1040, 528, False, 9, False)]
    want = [u16(c.call()) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                outs.append(c.call())
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            np.testing.assert_array_equal(u16(o), w)


# ---- the whole path --------------------------------------------------------------------


def _path(kind, x, ids, count, rw, w1, s1, w2, s2, idx, buf, out):
    """Routing map to layer output: mask and indices, dispatch, both products, combine."""
    e, k = w1.shape[0], ids.shape[1]
    mod.moe_mask_create_indices(ids, count, 0, e, idx["token_expert_order"], idx["expert_start_indices"],
                                idx["restore_token_order"], idx["expert_ids"], idx["expert_usage_stats"],
                                idx["workspace"])
    starts, active = idx["expert_start_indices"], idx["expert_ids"]
    if kind == "f8":
        mod.moe_dispatch_f8(x, k, idx["restore_token_order"], buf["a"], buf["sa"])
        mod.moe_expert_matmul_f8(buf["a"], buf["sa"], starts, active, w1, s1, buf["h"], flags=mod.MATMUL_SWIGLU)
        mod.moe_quantize_f8(buf["h"], buf["hq"], buf["sh"], row_count=starts[-1:])
        mod.moe_expert_matmul_f8(buf["hq"], buf["sh"], starts, active, w2, s2, buf["y"])
    else:
        mod.moe_dispatch(x, k, idx["restore_token_order"], buf["a"])
        mod.moe_expert_matmul(buf["a"], starts, active, w1, buf["h"], flags=mod.MATMUL_SWIGLU)
        mod.moe_expert_matmul(buf["h"], starts, active, w2, buf["y"])
    mod.moe_combine(buf["y"], rw, idx["restore_token_order"], k, out)


def _path_want(kind, x, ids, real, rw, w1, s1, w2, s2, e, h, i):
    """(out, bound) of the path in 64 bits with the roundings between the calls, and what fp32 may add to each."""
    halves = [(w1, s1, 2, i), (w2, s2, 1, h)]
    fw = []
    for w, s, n_halves, n in halves:
        v = f64(w)
        fw.append(v if s is None else np.stack([oracle.block_weights(v[a], s[a].cpu().numpy(), n_halves)
                                                for a in range(e)]))
    xv = f64(x)
    if kind == "f8":
        q, s = oracle.quantize_f8(u16(x))
        xv = oracle.e4m3_values()[q] * s[:, np.arange(h) // 128]
    out, bound = np.zeros((x.shape[0], h)), np.zeros((x.shape[0], h))
    for t in range(real):
        for j in range(ids.shape[1]):
            a = int(ids[t, j])
            if not 0 <= a < e:
                continue
            act, d_act = oracle.products(xv[t:t + 1], fw[0][a], True, kind == "f8")
            if kind == "f8":  # half a step of e4m3 of the value, of the block's largest 2^-9 / 448 below; the scale
                big = np.abs(act).reshape(-1)
                top = np.array([big[128 * b:128 * b + 128].max() for b in range(blocks(i))])[np.arange(i) // 128]
                d_act = d_act * 1.1 + (np.abs(act) + d_act) * 2.0 ** -4 * 1.01 + (top + d_act.max()) * 2.0 ** -10 / 448
            y, d_y = oracle.products(act, fw[1][a], False, kind == "f8")
            d_y = d_y + np.abs(fw[1][a]).dot(d_act[0]) * 1.01
            w = abs(float(rw[t, j]))
            out[t] += float(rw[t, j]) * y[0]
            bound[t] += w * (d_y[0] + np.abs(y[0]) * 2.0 ** -21)
    return out, bound + 2.0 ** -8 * (np.abs(out) + bound) + TINY


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("n, real, k, e, h, i", [(60, 41, 2, 4, 272, 400), (400, 400, 2, 3, 144, 80)])
def test_path_eager_and_replayed(kind, n, real, k, e, h, i):
    say("path", kind, n, h, i)
    g = torch.Generator(device=DEV).manual_seed(n)
    data = []
    for _ in range(3):
        ids = torch.stack([torch.randperm(e, generator=g, device=DEV)[:k] for _ in range(n)]).int()
        data.append((torch.randn((n, h), generator=g, device=DEV).to(torch.bfloat16), ids,
                     torch.softmax(torch.randn((n, k), generator=g, device=DEV), 1)))
    if kind == "f8":
        def weights(rows, depth, n_halves, per):
            return ((torch.randn((e, rows, depth), generator=g, device=DEV) * 105).clamp(-448, 448).to(F8),
                    (0.5 + torch.rand((e, n_halves * blocks(per), blocks(depth)), generator=g, device=DEV)) /
                    (105 * depth ** 0.5))
        (w1, s1), (w2, s2) = weights(2 * i, h, 2, i), weights(h, i, 1, h)
    else:
        w1 = (torch.randn((e, 2 * i, h), generator=g, device=DEV) * h ** -0.5).to(torch.bfloat16)
        w2 = (torch.randn((e, h, i), generator=g, device=DEV) * i ** -0.5).to(torch.bfloat16)
        s1 = s2 = None
    idx = mod.alloc_indices(n * k, e, DEV)
    buf = dict(h=torch.zeros((n * k, i), dtype=torch.bfloat16, device=DEV),
               y=torch.zeros((n * k, h), dtype=torch.bfloat16, device=DEV))
    if kind == "f8":
        buf["a"], buf["sa"] = mod.alloc_quantized_f8(n * k, h, DEV)
        buf["hq"], buf["sh"] = mod.alloc_quantized_f8(n * k, i, DEV)
    else:
        buf["a"] = mod.alloc_dispatch(n * k, h, DEV)
    x, ids, rw = (t.clone() for t in data[0])
    count, out = dev(np.array([real], np.int32)), torch.zeros((n, h), dtype=torch.bfloat16, device=DEV)
    eager = []
    for dx, dids, drw in data:
        x.copy_(dx), ids.copy_(dids), rw.copy_(drw)
        _path(kind, x, ids, count, rw, w1, s1, w2, s2, idx, buf, out)
        eager.append(u16(out))
        want, bound = _path_want(kind, dx, dids.cpu().numpy(), real, drw.cpu().numpy(), w1, s1, w2, s2, e, h, i)
        bad = ~(np.abs(f64(out) - want) <= bound)
        assert not bad.any(), (np.argwhere(bad)[:4], f64(out)[bad][:4], want[bad][:4], bound[bad][:4])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _path(kind, x, ids, count, rw, w1, s1, w2, s2, idx, buf, out)
    for turn in range(6):
        dx, dids, drw = data[turn % 3]
        x.copy_(dx), ids.copy_(dids), rw.copy_(drw)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(u16(out), eager[turn % 3])


def test_rows_on_two_streams_and_the_least_alignment():
    """Rows quantised from tensors that begin in the middle of their memory, on two streams at once."""
    g = np.random.default_rng(31)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = []
    for n, h in ((700, 7168), (33, 1040)):
        xb = _f8_rows(g, n, h)
        wq, ws = oracle.quantize_f8(xb)
        q, s = mod.alloc_quantized_f8(n, h, DEV)
        q.view(torch.uint8).fill_(77), s.fill_(-3.0)
        work.append((_moved(bf16_from_bits(xb, DEV), 8), _moved(q, 16), _moved(s, 1), wq, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for (x, q, s, _, _), stream in zip(work, streams):
            q.view(torch.uint8).fill_(77)
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                mod.moe_quantize_f8(x, q, s)
        torch.cuda.synchronize()
        for _, q, s, wq, ws in work:
            np.testing.assert_array_equal(codes(q), wq)
            np.testing.assert_array_equal(s.cpu().numpy(), ws)


# ---- refusals of tensors on the device ---------------------------------------------------


def _calls():
    """name -> (function, good keyword arguments)."""
    n, h, e, o = 8, 144, 3, 272
    x = torch.zeros((n, h), dtype=torch.bfloat16, device=DEV)
    q, s = mod.alloc_quantized_f8(n, h, DEV)
    starts, ids = u32_of([0, 2, 8, 8]), dev(np.array([0, 2, -1], np.int32))
    w, out = torch.zeros((e, o, h), dtype=torch.bfloat16, device=DEV), torch.zeros((n, o), dtype=torch.bfloat16, device=DEV)
    wq, sw = w.to(F8), torch.ones((e, blocks(o), blocks(h)), device=DEV)
    i = 48
    gu, d = torch.zeros((e, 2 * i, h), device=DEV).to(F8), torch.zeros((e, h, i), device=DEV).to(F8)
    return {
        "quantize": (mod.moe_quantize_f8, dict(x=x, out_q=q, out_scales=s, row_count=u32_of([3]))),
        "dispatch": (mod.moe_dispatch_f8, dict(input_tokens=x, top_k=2, restore_token_order=u32_of(np.arange(2 * n)),
                                               out_q=q, out_scales=s)),
        "matmul": (mod.moe_expert_matmul, dict(a=x, expert_start_indices=starts, expert_ids=ids, w=w, out=out, flags=0)),
        "matmul_f8": (mod.moe_expert_matmul_f8, dict(a_q=q, a_scales=s, expert_start_indices=starts, expert_ids=ids,
                                                     w_q=wq, w_scales=sw, out=out, flags=0)),
        "layer": (mod.moe_layer_few, dict(
            x=x, topk_ids=torch.zeros((n, 2), dtype=torch.int64, device=DEV), router_weights=torch.ones((n, 2), device=DEV),
            w_gate_up=gu, w_down=d, output_tokens=torch.zeros_like(x), workspace=mod.alloc_layer_few(n, 2, i, DEV),
            gate_up_scales=torch.ones((e, 2, 2), device=DEV), down_scales=torch.ones((e, 2, 1), device=DEV),
            real_token_count=dev(np.array([5], np.int32)), tp_rank=0)),
    }


@pytest.mark.parametrize("call", ["quantize", "dispatch", "matmul", "matmul_f8", "layer"])
def test_each_tensor_is_checked(call):
    fn, good = _calls()[call]
    fn(**good)
    for name, v in good.items():
        if not isinstance(v, torch.Tensor):
            continue
        for bad, error in ((v.cpu(), ValueError), (None, (TypeError, ValueError, AttributeError)), (v.to(torch.float64), TypeError),
                           (v.view(torch.uint8) if v.dtype != torch.uint8 else v.view(torch.int8), TypeError),
                           (torch.stack((v, v), -1)[..., 0] if v.numel() > 1 else None, ValueError),
                           (v.reshape(-1)[:-1] if v.numel() > 1 else v.expand(1).repeat(2), (ValueError, mod.MoeError)),
                           (torch.cat((v, v)), (ValueError, mod.MoeError))):
            optional = bad is None and name in ("row_count", "real_token_count")
            larger = name == "workspace" and isinstance(bad, torch.Tensor) and bad.dtype == torch.uint8 and bad.is_cuda \
                and bad.is_contiguous() and bad.numel() >= v.numel()
            if optional or larger or (bad is None and v.numel() == 1):
                continue
            with pytest.raises(error):
                fn(**{**good, name: bad})
    torch.cuda.synchronize()


def test_bad_numbers_are_refused():
    calls = _calls()
    for call, name, values in (("dispatch", "top_k", (0, -1, 3, 1025, 2 ** 40)), ("matmul", "flags", (2, 2 ** 33 + 2)),
                               ("matmul_f8", "flags", (2, 4, 2 ** 33 + 2)), ("layer", "tp_rank", (-1,))):
        fn, good = calls[call]
        for v in values:
            with pytest.raises((ValueError, mod.MoeError, OverflowError)):
                fn(**{**good, name: v})
    fn, good = calls["matmul_f8"]
    with pytest.raises(ValueError):  # SwiGLU: the weights' scales are two halves of blocks
        fn(**{**good, "flags": mod.MATMUL_SWIGLU})
    with pytest.raises(ValueError):
        calls["layer"][0](**{**calls["layer"][1], "gate_up_scales": None, "down_scales": None})


def test_no_rows():
    """Buffers without rows, and groups without rows: nothing to do, nothing written."""
    calls = _calls()
    empty = torch.zeros((0, 144), dtype=torch.bfloat16, device=DEV)
    q, s = mod.alloc_quantized_f8(0, 144, DEV)
    mod.moe_quantize_f8(empty, q, s)
    mod.moe_dispatch_f8(empty, 2, u32_of([]), q, s)
    g = calls["matmul_f8"][1]
    none = torch.zeros((0, 272), dtype=torch.bfloat16, device=DEV)
    mod.moe_expert_matmul_f8(q, s, g["expert_start_indices"], g["expert_ids"], g["w_q"], g["w_scales"], none)
    mod.moe_expert_matmul(empty, g["expert_start_indices"], g["expert_ids"], calls["matmul"][1]["w"], none)
    l = dict(calls["layer"][1])
    for name in ("x", "topk_ids", "router_weights", "output_tokens"):
        l[name] = l[name][:0]
    mod.moe_layer_few(**l)
    out = torch.full((8, 272), 7.0, dtype=torch.bfloat16, device=DEV)
    for name in ("matmul", "matmul_f8"):
        calls[name][0](**{**calls[name][1], "expert_start_indices": u32_of([0, 0, 0, 0]), "out": out})
    assert (out == 7.0).all()
