"""The logits' gradient for choices that routing would not have made: of no expert, and
of logits that are not numbers."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref
from tests.test_gpu_train_columns import INF, NAN, same
from tests.test_gpu_train_router import EPS, backward64, logits_of

pytestmark = pytest.mark.gpu


def of(experts):
    """A routing of these experts."""
    return (None, experts.to("cuda", torch.int32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_what_no_choice_carries_is_not_read(renormalize, dtype):
    """NaN and infinities at -1, at experts out of range, and at logits of -infinity and NaN."""
    tokens, experts, top_k = 200, 72, 6
    l = logits_of(tokens, experts, 1, dtype)
    g = torch.Generator(device="cuda").manual_seed(2)
    chosen = torch.rand(tokens, experts, generator=g, device="cuda").argsort(1)[:, :top_k].int()
    chosen[:, 5] = torch.tensor([-1, experts, 1 << 30, -(1 << 31)], device="cuda").repeat(50)
    chosen[::3, 2:] = -1
    chosen[::7] = -1
    l[torch.arange(1, tokens, 5), chosen[1::5, 1].clamp(min=0).long()] = -INF
    l[torch.arange(2, tokens, 5), chosen[2::5, 1].clamp(min=0).long()] = NAN
    none = (chosen < 0) | (chosen >= experts)
    at = torch.gather(l, 1, torch.where(none, 0, chosen).long()).float()
    none |= ~(at > -INF)
    dw = torch.randn(tokens, top_k, generator=g, device="cuda")
    slopes = torch.randn(experts, generator=g, device="cuda")
    want, mag = backward64(l, torch.where(none, -1, chosen), dw, slopes, renormalize)
    clean = fg.moe_route_backward(l, of(chosen), torch.where(none, 0.0, dw), slopes, renormalize=renormalize)
    ref.within(clean, want, ref.REL * mag + EPS[dtype] * want.abs() + 1e-38)
    for odd in (NAN, INF, -INF):
        same(fg.moe_route_backward(l, of(chosen), torch.where(none, odd, dw), slopes, renormalize=renormalize), clean)
