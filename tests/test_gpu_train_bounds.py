"""Bounds that include/fg.h gives for 32-bit results: of the gated activation's
gradient, whose sigmoid comes from fast functions, and of sums under 2^-126."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref
from tests.test_gpu_train_columns import same

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a unit of a 32-bit value's last place, relative


@pytest.mark.parametrize("mode", ref.MODES)
def test_sigmoid(mode):
    """du = g s dy for every gate that e4m3 has, over scales of 2^-8 .. 2: s within (10 + 1.3 |g|) U of itself where g is
    negative, and within 10 U elsewhere.  exp(-g)'s exponent g log2(e) is off by the product's rounding, U, and the
    constant's, 0.22 U, of itself, and so exp(-g) by 1.22 |g| U; its power by 4 U, the sum by U, the reciprocal by 2 U,
    the two products of du by U each.  Above g = 0 the error of exp(-g) counts by exp(-g) / (1 + exp(-g)), whose product
    with 1.22 g is under 0.35."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes = codes[(codes & 0x7f) != 0x7f].view(torch.float8_e4m3fn).float()
    g = torch.cat([codes * 2.0 ** k for k in range(-8, 2)])
    g = g[(g > -87) & (g < 1000)]
    n = (g.numel() + 127) // 128 * 128
    g = torch.cat([g, g.new_ones(n - g.numel())])
    x = torch.ones(n, 256, device="cuda")
    x[:, :128] = g[:, None]
    saved, scales = fg.quantize(mode, x)
    v = ref.decoded(saved, scales)[:, :128]
    d = fg.swiglu_backward(mode, torch.ones(n, 128, device="cuda"), saved, scales, plain=True)
    want = v * torch.sigmoid(v)
    ref.within(d.dx[:, 128:], want, (10 + 1.3 * (-v).clamp(min=0)) * U * want.abs() + 2.0 ** -149)


def test_sums_of_weight_gradients_under_the_smallest_normal_number():
    """accumulate may take sums and addends under 2^-126 for zero, and nothing else."""
    offsets = ref.fixed_offsets([64, 0])
    a = fg.quantize_columns(torch.zeros(64, 128, device="cuda"), offsets)
    b = fg.quantize_columns(torch.ones(64, 128, device="cuda"), offsets)
    out = torch.empty(2, 128, 128, device="cuda")
    kept = torch.cat([torch.ldexp(torch.ones(64, device="cuda"), torch.arange(-140, -76, device="cuda")),
                      -torch.ldexp(torch.ones(64, device="cuda"), torch.arange(-140, -76, device="cuda"))])
    out[:] = kept
    fg.grouped_wgrad(a, b, offsets, out=out, accumulate=True)
    ref.within(out[0], kept.double().expand(128, 128), torch.full((128, 128), 2.0 ** -126, dtype=torch.float64, device="cuda"))
    normal = kept.abs() >= 2.0 ** -126
    same(out[0][:, normal], kept[normal].expand(128, -1))
    same(out[1], kept.expand(128, 128))  # no rows: left as it was
