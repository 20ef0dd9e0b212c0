"""fp8_block128's scale where its quotient has few bits left, or none.

The scale amax / 448 of a block of least values is rounded up, so that it is
never zero and no code saturates.  In units of 2^-149 (the least fp32 value) a
block of whole numbers up to n < 2^17 has the scale ceil(n / 448); one above
2^17 the nearest.
"""
import numpy as np
import pytest
import torch

import inputs
import mx_gemm_gb300 as fg
import oracle
from tests.test_gpu_quantize import decoded

pytestmark = pytest.mark.gpu


def from_ulps(n):
    """fp32 values n * 2^-149 of whole numbers |n| < 2^23."""
    n = np.asarray(n, np.int64)
    return np.where(n < 0, np.abs(n) | 0x80000000, n).astype(np.uint32).view(np.float32)


TINY = [1, 2, 71, 223, 224, 225, 447, 448, 449, 464, 465, 671, 672, 673, 895, 1000, 7135, 100_000, (1 << 17) - 1, 300_000]


def test_tiny_blocks_beside_zeros():
    k = 256
    x = np.zeros((len(TINY), k), np.int64)
    rng = np.random.default_rng(1)
    for i, n in enumerate(TINY):
        x[i, :128:2] = rng.integers(-n, n + 1, 64)
        x[i, 6] = n if i % 2 else -n
        x[i, 130] = n                       # one value in a block of zeros
    codes, scales = fg.quantize("fp8_block128", torch.from_numpy(from_ulps(x)).cuda())
    amax = np.abs(x.reshape(-1, 2, 128)).max(axis=2)
    s = from_ulps(np.where(amax < 1 << 17, -(-amax // 448), np.rint(amax / 448).astype(np.int64)))
    assert np.array_equal(scales.cpu().numpy(), s)
    q = (from_ulps(x).reshape(-1, 2, 128) / s[:, :, None]).reshape(x.shape)
    assert np.array_equal(decoded(codes, "fp8_block128"), oracle.table_e4m3()[inputs.to_e4m3_codes(q)])


def test_tiny_blocks_in_a_product():
    """Finite operands give finite products: a row whose values underflow adds nothing."""
    x = torch.zeros(4, 256)
    x[0, 3] = 1e-45
    x[1, 5] = 1e-43
    x[2] = 1.0
    x[2, 128] = 1.0
    x[2, 129:] = 0
    a, a_s = fg.quantize("fp8_block128", x.cuda())
    g = torch.Generator().manual_seed(1)
    b = torch.randn(128, 256, generator=g).to(torch.float8_e4m3fn).cuda()
    b_s = torch.ones(1, 2, device="cuda")
    pb = fg.preshuffle_b("fp8_block128", b, b_s)
    offsets = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for y in (fg.gemm(a, pb, a_s), fg.grouped_gemm(a, pb, offsets, a_s)):
        assert torch.isfinite(y).all() and (y[[0, 1, 3]].float().abs() < 1e-30).all() and (y[2] != 0).any()


def test_tiny_blocks_of_a_norm():
    """The norm's output quantises the same way: x = 1 with a weight of least values beside zeros."""
    w = np.zeros(256, np.int64)
    w[3], w[200], w[201] = 100, 1, -1
    codes, scales, _, y = fg.rmsnorm_quantize("fp8_block128", torch.ones(2, 256, device="cuda"),
                                              torch.from_numpy(from_ulps(w)).cuda(), eps=0.0, normed=True)
    n = y.cpu().numpy()
    assert np.array_equal(scales.cpu().numpy(), np.tile(from_ulps([1, 1]), (2, 1)))
    assert np.array_equal(decoded(codes, "fp8_block128"),
                          oracle.table_e4m3()[inputs.to_e4m3_codes((n / from_ulps(1)).astype(np.float32))])
