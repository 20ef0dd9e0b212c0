"""Arguments of the compiled binding that are no tensors."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests.test_gpu_grouped import Experts

WIDE = 1 << 32


@pytest.mark.parametrize("value", [WIDE + 1, -WIDE + 1, 1 << 31, 1 << 70])
def test_integers_that_do_not_fit(value):
    """2^32 + 1 is not 1: act = 1 reads rows of twice the columns, a mode sizes the outputs."""
    fg.moe.binding()
    x = torch.zeros(4, 256, dtype=torch.bfloat16)  # refused before the tensor, which is not on a GPU, is looked at
    with pytest.raises(ValueError, match="act"):
        fg.quantize("mxfp8_b32", x, act=value)
    with pytest.raises(ValueError, match="mode"):
        fg.quantize(value, x)
    with pytest.raises(ValueError, match="mode"):
        fg.rmsnorm_quantize(value, x, x[0])


@pytest.mark.gpu
@pytest.mark.parametrize("value", [WIDE, -1, WIDE + (1 << 30)])
def test_flags_that_do_not_fit(value):
    c = Experts("mxfp8_b32", [4, 4, 4], 128, 256, 1)
    with pytest.raises(ValueError, match="flags"):
        c.run(flags=value)


class NoTruth:
    def __bool__(self):
        raise TypeError("neither")


@pytest.mark.gpu
def test_values_without_a_truth_value():
    x = torch.randn(4, 256, device="cuda")
    with pytest.raises(ValueError, match="renormalize"):
        fg.moe_route(x, 2, renormalize=NoTruth())
    with pytest.raises(ValueError, match="normed"):
        fg.rmsnorm_quantize("mxfp8_b32", x, x[0].contiguous(), normed=NoTruth())
    assert fg.moe_route(x, 2, renormalize=1).experts.shape == (4, 2)
