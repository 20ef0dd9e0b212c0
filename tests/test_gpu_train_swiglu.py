"""The gated activation's backward pass from its 8-bit checkpoint.

Codes and scales are held to the 64-bit formula of the values that the checkpoint
stands for: each value within half a step of e4m3 and the 32-bit arithmetic's
error (train_ref.near).  The plain gradient: within that error, and half a step of
its type.  The routing weights' gradient: the error of each product, and 2^-24 of
the magnitudes' sum for each of the additions.
"""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref
from tests.test_gpu_train_columns import INF, NAN, rand, same

pytestmark = pytest.mark.gpu

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
SMALL = 2.0 ** -134  # half a step of bf16's values below 2^-126, which are 2^-133 apart


def formula(dy, g, u, w):
    """fp64 (dg, du), act, dots and the magnitudes that their errors are measured by.

    exp(-g)'s exponent, -g log2(e), is rounded once: by up to 2^-24 of itself, which
    multiplies the result by up to 1 + 2^-24 |g| = 1 + REL |g| / 64.  Where s is under
    2^-126 = REL 2^-108 it counts as 0."""
    s = torch.sigmoid(g)
    rest = torch.sigmoid(-g)
    act = g * s * u
    dg = w * dy * u * s * (1 + g * rest)
    du = w * dy * g * s
    mag = torch.cat([(w * dy * u * s).abs() * (1 + (g * rest).abs()), du.abs()], dim=1)
    mag = mag * (1 + g.abs().repeat(1, 2) / 64) + (w * dy * (1 + g.abs()) * (1 + u.abs())).abs().repeat(1, 2) * 2.0 ** -108
    return torch.cat([dg, du], dim=1), mag, act, (dy * act)


def act_mag(g, u, w=1.0):
    """The magnitude for w * act, likewise."""
    return (w * (g * torch.sigmoid(g) * u)).abs() * (1 + g.abs() / 64) + w * (g * u).abs() * 2.0 ** -108


def slot_weights(r, rows):
    w = torch.zeros(rows, dtype=torch.float64, device="cuda")
    ok = r.slots >= 0
    w[r.slots[ok].long()] = r.weights[ok].double()
    return w


@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,width", [(1, 128), (33, 256), (128, 384), (1000, 128)])
def test_without_routing(mode, dtype, rows, width):
    saved, scales = fg.quantize(mode, rand(1, rows, 2 * width))
    dy = (rand(2, rows, width) / 64).to(dtype)
    d = fg.swiglu_backward(mode, dy, saved, scales, columns=True, plain=True)
    v = ref.decoded(saved, scales)
    want, mag, act, _ = formula(dy.double(), v[:, :width], v[:, width:], 1.0)
    assert d.dweights is None and d.dx.dtype == dtype
    ref.within(d.dx, want, ref.REL * mag + EPS[dtype] * want.abs() + SMALL)
    ref.near(d.codes.double(), d.scales, want, mag, mode, "rows")
    for c, x, m in ((d.dx_columns, want, mag), (d.act_columns, act, act_mag(v[:, :width], v[:, width:]))):
        codes, s = ref.matrix(c)
        ref.near(codes, s, ref.by_place(x, [0, rows], rows), ref.by_place(m, [0, rows], rows), "columns", "columns")
    few = fg.swiglu_backward(mode, dy, saved, scales)
    assert few.dx is None and few.dx_columns is None and few.act_columns is None
    same(few.codes.view(torch.uint8), d.codes.view(torch.uint8))


@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("tokens,experts,top_k,width", [(1, 8, 2, 128), (61, 40, 8, 256), (300, 6, 3, 640), (515, 100, 1, 128)])
def test_with_routing(mode, tokens, experts, top_k, width):
    r, _ = ref.routing(tokens, experts, top_k, 3, padded=0.1 if tokens > 1 else 0.0, empty=(1, experts - 1))
    rows = tokens * top_k
    routed = int(r.offsets[-1])
    saved, scales = fg.quantize(mode, rand(4, rows, 2 * width))
    dy = (rand(5, rows, width) / 64).to(torch.bfloat16)
    dy[routed:] = NAN  # rows of no expert are not read
    d = fg.swiglu_backward(mode, dy, saved, scales, routing=r, columns=True, plain=True)
    v, w = ref.decoded(saved, scales), slot_weights(r, rows)[:, None]
    dy = torch.where(torch.arange(rows, device="cuda")[:, None] < routed, dy.double(), 0.0)
    want, mag, act, dots = formula(dy, v[:, :width], v[:, width:], w)
    ref.within(d.dx, want, ref.REL * mag + 2.0 ** -8 * want.abs() + SMALL)
    assert not d.codes.view(torch.uint8)[routed:].any() and not d.dx[routed:].any()
    assert (ref.scale_values(d.scales)[routed:] == 1).all()
    ref.near(d.codes.double(), d.scales, want, mag, mode, "rows")
    offsets = r.offsets.tolist()
    for c, x, m in ((d.dx_columns, want, mag), (d.act_columns, w * act, act_mag(v[:, :width], v[:, width:], w))):
        codes, s = ref.matrix(c)
        ref.near(codes, s, ref.by_place(x, offsets, rows), ref.by_place(m, offsets, rows), "columns", "columns")
    ok, at = r.slots >= 0, r.slots.clamp(min=0).long()
    want = torch.where(ok, dots.sum(1)[at], 0.0)
    bound = ((ref.REL + width * 2.0 ** -24) * dots.abs() + ref.REL * dy.abs() * act_mag(v[:, :width], v[:, width:])).sum(1)[at]
    ref.within(d.dweights, want, bound)
    assert (d.dweights[~ok] == 0).all()


@pytest.mark.parametrize("mode", ("mxfp8_b32", "mxfp4_fp8a"))
def test_widths_of_whole_32_blocks(mode):
    """Without columns a width need not be a multiple of 128."""
    for width in (32, 96, 160, 288):
        r, _ = ref.routing(50, 7, 2, 6, padded=0.1)
        saved, scales = fg.quantize("mxfp8_b32", rand(7, 100, 2 * width))
        dy = rand(8, 100, width)
        routed = int(r.offsets[-1])
        d = fg.swiglu_backward(mode, dy, saved, scales, routing=r, plain=True)
        v, w = ref.decoded(saved, scales), slot_weights(r, 100)[:, None]
        dy = torch.where(torch.arange(100, device="cuda")[:, None] < routed, dy.double(), 0.0)
        want, mag, _, dots = formula(dy, v[:, :width], v[:, width:], w)
        ref.within(d.dx, want, ref.REL * mag + 2.0 ** -24 * want.abs() + SMALL)
        ref.near(d.codes.double(), d.scales, want, mag, "mxfp8_b32", "rows")
        assert (d.codes.view(torch.uint8)[routed:] == 0).all() and (ref.scale_values(d.scales)[routed:] == 1).all()
        at = r.slots.clamp(min=0).long()
        ref.within(d.dweights, torch.where(r.slots >= 0, dots.sum(1)[at], 0.0),
                   ((2 * ref.REL + width * 2.0 ** -24) * dots.abs() + ref.REL * dy.abs() * act_mag(v[:, :width], v[:, width:])).sum(1)[at])
        with pytest.raises(fg.FgError):
            fg.swiglu_backward(mode, dy.float(), saved, scales, routing=r, columns=True)


def test_gates_from_one_end_to_the_other():
    """Gates of any size: 1 - s is exact where s is 1, s is 0 below -88.7."""
    gates = torch.tensor([0.0, 1e-30, -1e-30, 1.0, -1.278, 8.0, 17.0, 20.0, 88.0, 104.0, 448.0, -8.0, -17.0, -80.0, -87.0, -88.0,
                          -104.0, -448.0], device="cuda")
    x = torch.zeros(18 * 4, 256, device="cuda")
    for i, scale in enumerate((1.0, 2.0 ** 20, 2.0 ** 100, 2.0 ** -20)):
        x[18 * i:18 * i + 18, :128] = (gates * scale)[:, None]
        x[18 * i:18 * i + 18, 128:] = 2.0
    saved, scales = fg.quantize("mxfp8_b32", x)
    dy = torch.full((72, 128), 0.5, device="cuda")
    d = fg.swiglu_backward("mxfp8_b32", dy, saved, scales, plain=True)
    v = ref.decoded(saved, scales)
    want, mag, _, _ = formula(dy.double(), v[:, :128], v[:, 128:], 1.0)
    ref.within(d.dx, want, ref.REL * mag + 2.0 ** -24 * want.abs() + SMALL)
    assert torch.isfinite(d.dx).all()


def test_products_that_pass_32_bits_before_they_are_small():
    """dy * u is above every 32-bit number, its product with the activation's slope is not."""
    x = torch.empty(64, 256, device="cuda")
    x[:, :128] = torch.tensor([-28.0, -60.0, -80.0, -104.0], device="cuda").repeat(16)[:, None]
    x[:, 128:] = 2.0 ** 30
    saved, scales = fg.quantize("mxfp8_b32", x)
    dy = torch.full((64, 128), 2.0 ** 100, device="cuda")
    d = fg.swiglu_backward("mxfp8_b32", dy, saved, scales, plain=True)
    v = ref.decoded(saved, scales)
    want, mag, _, _ = formula(dy.double(), v[:, :128], v[:, 128:], 1.0)
    assert (dy.double() * v[:, 128:]).min() > 3.5e38
    ref.within(d.dx, want, ref.REL * mag + 2.0 ** -24 * want.abs() + SMALL)


def test_values_that_are_not_numbers_stay_within_their_blocks():
    x = rand(9, 64, 512)
    x[3, 5], x[40, 256 + 130] = NAN, INF
    saved, scales = fg.quantize("mxfp8_b32", x)
    dy = rand(10, 64, 256)
    dy[20, 200] = INF
    d = fg.swiglu_backward("mxfp8_b32", dy, saved, scales, columns=True)
    s = ref.scale_values(d.scales).view(64, 16)
    bad = torch.zeros(64, 16, dtype=torch.bool, device="cuda")
    bad[3, [0, 8]] = True                          # the checkpoint's block of (3, 5) is NaN: dg and du
    bad[40, 4] = True                              # u's block 4: dg alone
    bad[20, [6, 14]] = True                        # dy's value: both
    same(torch.isnan(s), bad)
    assert (d.codes.view(64, 16, 32).double()[bad] == 0).all()
    _, c = ref.matrix(d.act_columns)
    bad = torch.zeros_like(c, dtype=torch.bool)
    bad[0:32, 0] = True                            # act of row 3, columns 0..31
    bad[128:160, 1] = True                         # of row 40
    same(c == 255, bad)


def test_a_view_of_the_gradient():
    saved, scales = fg.quantize("mxfp8", rand(11, 50, 512))
    big = rand(12, 100, 700).to(torch.bfloat16)
    dy = big[::2, 8:264]
    a = fg.swiglu_backward("mxfp8", dy, saved, scales)
    b = fg.swiglu_backward("mxfp8", dy.contiguous(), saved, scales)
    same(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
    same(a.scales.view(torch.uint8), b.scales.view(torch.uint8))


def test_no_rows():
    saved, scales = fg.quantize("mxfp8_b32", rand(13, 2, 512)[:0])
    d = fg.swiglu_backward("mxfp8_b32", torch.empty(0, 256, device="cuda"), saved, scales, columns=True, plain=True)
    assert d.codes.shape == (0, 512) and d.dx_columns.K == 128 and not d.dx_columns.data.any()


def test_against_differences():
    """dg and du against central differences of the activation in 64 bits."""
    width, h = 128, 1e-5
    saved, scales = fg.quantize("mxfp8_b32", rand(14, 40, 2 * width, spread=False))
    dy = rand(15, 40, width, spread=False)
    d = fg.swiglu_backward("mxfp8_b32", dy, saved, scales, plain=True)
    v = ref.decoded(saved, scales)

    def loss(x):
        g, u = x[:, :width], x[:, width:]
        return dy.double() * (g * torch.sigmoid(g) * u)

    for part in (0, 1):
        step = torch.zeros_like(v)
        step[:, part * width:(part + 1) * width] = h
        num = (loss(v + step) - loss(v - step)) / (2 * h)
        got = d.dx[:, part * width:(part + 1) * width].double()
        # h^2 / 6 of a third derivative below 4 |dy u|, 1e-16 / h of rounding, and the arithmetic's error
        mag = dy.double().abs() * (1 + v.abs().amax()) ** 2
        ref.within(got, num, (4 * h * h + 1e-10 + ref.REL) * mag)


def test_refusals():
    r, _ = ref.routing(10, 4, 2, 16)
    saved, scales = fg.quantize("mxfp8_b32", rand(17, 20, 512))
    dy = rand(18, 20, 256)
    for call, match in [
            (lambda: fg.swiglu_backward("mxfp8_b32", dy, saved, scales[:, :8].contiguous()), "scales"),
            (lambda: fg.swiglu_backward("mxfp8", dy, saved, scales), "scales"),
            (lambda: fg.swiglu_backward("fp8_block128", dy, saved, scales), "dtype"),
            (lambda: fg.swiglu_backward("mxfp8_b32", dy[:10], saved, scales), "shape"),
            (lambda: fg.swiglu_backward("mxfp8_b32", dy.half(), saved, scales), "dtype"),
            (lambda: fg.swiglu_backward("mxfp8_b32", dy.T, saved, scales), "contiguous"),
            (lambda: fg.swiglu_backward("mxfp8_b32", dy[:18], saved[:18], scales[:18], routing=r), "routing"),
            (lambda: fg.swiglu_backward("mxfp8_b32", dy, saved.cpu(), scales), "CUDA")]:
        with pytest.raises(ValueError, match=match):
            call()
