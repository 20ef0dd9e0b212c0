"""The gated activation silu(g) u = g / (1 + exp(-g)) u at the ends of 32 bits.

Gates down to -88.7, the end of fp32's exp(-g), are held to the 64-bit value.
The arithmetic: the exponent -g log2(e) is rounded once, and its constant
once, (2^-24 + 2^-25) |g| < 2^-17 of the value together; the fast power, the
sum, the reciprocal and the products add less than 2^-20.  REL covers both.
"""
import numpy as np
import pytest
import torch

import inputs
import mx_gemm_gb300 as fg
from tests.test_gpu_quantize import block, code_bytes, decoded

pytestmark = pytest.mark.gpu

REL = 2.0 ** -16


def gated(x):
    g, u = np.split(x, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def assert_stands_for(codes, scales, want, mode):
    """Scales are those of `want`, or of a value REL away; values are within half a step of it."""
    b = block(mode)
    amax = np.abs(want.reshape(want.shape[0], -1, b)).max(axis=2)
    if mode == "fp8_block128":
        s = scales.cpu().double().numpy()
        assert (np.abs(s - amax / 448) <= (REL + 2.0 ** -23) * amax / 448).all()
    else:
        c = code_bytes(scales).astype(np.int64)
        top = inputs.E2M1_MAX if mode == "mxfp4" else inputs.E4M3_MAX
        lo, hi = (inputs.e8m0_for(amax * f, top).astype(np.int64) for f in (1 - REL, 1 + REL))
        assert ((c >= lo) & (c <= hi)).all()
        s = np.ldexp(1.0, c - 127)
    s = np.repeat(s, b, axis=1)
    man, low = (1, 0) if mode == "mxfp4" else (3, -6)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(want) / s, 1e-300))), low)
    half = np.ldexp(0.5, (e - man).astype(np.int64)) * s
    assert (np.abs(decoded(codes, mode) * s - want) <= half * (1 + 2.0 ** -10) + REL * np.abs(want)).all()


MODES = ("mxfp8_b32", "mxfp8", "mxfp4", "fp8_block128")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gates_near_the_end_of_exp(mode, dtype):
    """Gates from -88.5 to -80 against factors that bring the product back into the middle of the range."""
    g = torch.Generator().manual_seed(3)
    x = torch.empty(24, 1024)
    x[:, :512] = -80 - 8.5 * torch.rand(24, 512, generator=g)
    x[:, 512:] = torch.randn(24, 512, generator=g) * 10.0 ** torch.randint(5, 30, (24, 1), generator=g).float()
    x[3, :512] = -88.0                          # whole blocks past the reciprocal's least normal value
    x[4, :512] = -87.5
    x[5, 0::2] = -88.5                          # ... and beside others
    x = x.to(dtype)
    codes, scales = fg.quantize(mode, x.cuda(), act="swiglu")
    assert_stands_for(codes, scales, gated(x.double().numpy()), mode)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 128), (17, 2048), (300, 1408)])
def test_gated_activation_in_fp8_block128(dtype, m, k):
    g = torch.Generator().manual_seed(m + k)
    x = (3 * torch.randn(m, 2 * k, generator=g)).to(dtype)
    codes, scales = fg.quantize("fp8_block128", x.cuda(), act="swiglu")
    assert_stands_for(codes, scales, gated(x.double().numpy()), "fp8_block128")


def test_gates_of_any_size_with_ordinary_factors():
    """The largest and least gates keep their value: no product on the way leaves the range."""
    x = torch.zeros(6, 256)
    x[0, :128], x[0, 128:] = 3e38, 1.0
    x[1, :128], x[1, 128:] = 3e38, 1e-30
    x[2, :128], x[2, 128:] = 1e-38, 1.0
    x[3, :128], x[3, 128:] = 1e-38, 1e38
    x[4, :128], x[4, 128:] = -1e-37, -3e38
    x[5, :128], x[5, 128:] = -3e38, 1.0         # silu is zero
    codes, scales = fg.quantize("mxfp8", x.cuda(), act="swiglu")
    want = gated(x.double().numpy())
    assert_stands_for(codes[:5], scales[:5], want[:5], "mxfp8")
    assert (code_bytes(codes[5:]) & 0x7f == 0).all() and (code_bytes(scales[5:]) == 127).all()
