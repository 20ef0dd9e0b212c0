"""fp8_block128's codes are the quotients v / s rounded once, whatever way they are
worked out: at block scales near the smallest ones, where a remainder is no longer
exact, and for zeros, which keep their sign."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref
from tests.test_gpu_train_columns import rand, same

pytestmark = pytest.mark.gpu

MODE = "fp8_block128"


def quotients(v, s):
    """Bytes of the codes of 32-bit v / s, tensor by tensor: rounded once."""
    return (v / s).to(torch.float8_e4m3fn).view(torch.uint8)


def near_borders(exponent):
    """Rows of 128 values whose quotients by their block's scale lie at and next to borders between codes; the
    scales' last bits are those where a remainder's are lost first: near 1, 1.5 and 2 times 2^exponent."""
    m = torch.cat([torch.arange(a, b) for a, b in ((0x800000, 0x800040), (0xbfffc0, 0xc00040), (0xfffe00, 0x1000000))])
    s = torch.ldexp(m.double(), torch.tensor(exponent - 23))
    rows = torch.zeros(m.numel(), 128)
    rows[:, 0] = (448 * s).float()
    at = 1
    for border in (1, 3, 5, 7, 17 * 16, 19 * 16, 21 * 1024, 29 * 8192):
        for ulps in (-2, -1, 0, 1, 2, 3):
            v = ((s * border * 2.0 ** -10).float().view(torch.int32) + ulps).view(torch.float32)
            rows[:, at], rows[:, at + 1] = v, -v
            at += 2
    return rows


@pytest.mark.parametrize("exponent", list(range(-104, -86)) + [-30, 0, 97, 98, 99, 100, 101, 110])
def test_next_to_borders_between_codes(exponent):
    x = near_borders(exponent).cuda()
    s = torch.where(x[:, 0] == 0, torch.ones_like(x[:, 0]), ref.over_448(x.abs().amax(1).double()).float())[:, None]
    want = quotients(x, s)
    codes, scales = fg.quantize(MODE, x)
    same(scales, s)
    same(codes.view(torch.uint8), want)
    y = torch.cat([x, x], 1)
    _, _, saved, saved_scales = fg.swiglu_checkpoint(MODE, y)
    same(saved.view(torch.uint8), torch.cat([want, want], 1))
    # weights: a row's values over a block
    w = torch.zeros(x.shape[0], 128, 128, device="cuda")
    w[:, 5] = x
    for transpose in (False, True):
        codes, scales = fg.quantize_weight(MODE, w, transpose=transpose)
        got = codes.view(-1, 128, 128)
        same(scales.view(-1, 1), s)
        same((got[:, :, 5] if transpose else got[:, 5]).reshape(x.shape).view(torch.uint8), want)
    # and the rows of the activation's gradient: gates of 88 and values of 1 leave dg near dy
    saved, saved_scales = fg.quantize(MODE, torch.cat([torch.full_like(x, 88.0), torch.ones_like(x)], 1))
    d = fg.swiglu_backward(MODE, x, saved, saved_scales, plain=True)
    same(d.codes.view(torch.uint8), quotients(d.dx, d.scales.repeat_interleave(128, 1)))


def with_zeros(seed, *shape):
    """Values among which are zeros of either sign, and blocks of nothing else."""
    x = rand(seed, *shape)
    g = torch.Generator(device="cuda").manual_seed(seed)
    where = torch.rand(shape, generator=g, device="cuda")
    x = torch.where(where < 0.2, 0.0, torch.where(where < 0.4, -0.0, x))
    x.view(-1, x.shape[-1])[:128, :128] = -0.0
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [0, 110, -110])
def test_zeros_keep_their_sign(size, dtype):
    x = torch.ldexp(with_zeros(1, 256, 512), torch.tensor(size, device="cuda")).to(dtype)
    assert torch.signbit(x[0, 0]) and not x[0, 0]
    codes, scales = fg.quantize(MODE, x)
    want = quotients(x.float(), scales.repeat_interleave(128, 1))
    same(codes.view(torch.uint8), want)
    _, _, saved, _ = fg.swiglu_checkpoint(MODE, x)
    same(saved.view(torch.uint8), want)
    for transpose in (False, True):
        codes, scales = fg.quantize_weight(MODE, x, transpose=transpose)
        v = (x.T if transpose else x).float()
        same(codes.view(torch.uint8), quotients(v, scales.repeat_interleave(128, 0).repeat_interleave(128, 1)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_of_the_norm_and_the_activation_keep_their_sign(dtype):
    x = with_zeros(2, 256, 512).to(dtype)
    codes, scales, _, y = fg.rmsnorm_quantize(MODE, x, torch.ones(512, device="cuda", dtype=dtype), normed=True)
    zero = y == 0
    assert torch.signbit(y[zero]).any() and not torch.signbit(y[zero]).all()
    same(codes.view(torch.uint8)[zero], torch.where(torch.signbit(y[zero]), 0x80, 0).to(torch.uint8))
    # gate 0 or -0, and value 0 or -0: the product's sign is that of either
    codes, _ = fg.quantize(MODE, x, act="swiglu")
    g, u = x.float().chunk(2, 1)
    zero = (g == 0) | (u == 0)
    sign = torch.signbit(g) ^ torch.signbit(u)
    same(codes.view(torch.uint8)[zero], torch.where(sign[zero], 0x80, 0).to(torch.uint8))


def test_zeros_of_the_gradient_keep_their_sign():
    dy = with_zeros(3, 256, 256)
    saved, saved_scales = fg.quantize(MODE, rand(4, 256, 512))
    d = fg.swiglu_backward(MODE, dy, saved, saved_scales, plain=True)
    assert torch.signbit(d.dx[d.dx == 0]).any() and not torch.signbit(d.dx[d.dx == 0]).all()
    same(d.codes.view(torch.uint8), quotients(d.dx, d.scales.repeat_interleave(128, 1)))


def test_blocks_that_hold_no_number_have_codes_of_zero():
    x = rand(5, 8, 256)
    x[2, 5], x[3, 200] = float("nan"), -float("inf")
    codes, scales = fg.quantize(MODE, x)
    bad = torch.isnan(scales)
    assert bad.tolist() == [[i == 2, i == 3] for i in range(8)]
    assert not codes.view(torch.uint8).view(8, 2, 128)[bad].any()
    w = x.repeat(16, 1)
    w[:, 128:] = w[:, 128:].nan_to_num(posinf=1.0, neginf=1.0)
    for transpose in (False, True):
        codes, scales = fg.quantize_weight(MODE, w, transpose=transpose)
        assert int(torch.isnan(scales).sum()) == 1 and torch.isnan(scales.view(-1)[0])
        assert not codes.view(torch.uint8)[:128, :128].any()
