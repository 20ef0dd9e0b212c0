"""The logits' gradient for choices that routing would not have made: of no expert, of
logits that are not numbers, and far below the token's largest logit."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("below", [0.0, 90.0, 103.0, 150.0, 1e30])
def test_choices_far_below_the_largest_logit(below, dtype):
    """Renormalised weights are the softmax of the chosen logits alone, however far the largest one is."""
    tokens, experts, top_k = 60, 40, 4
    l = logits_of(tokens, experts, 3).to(dtype)
    l[:, 10:20] += below
    g = torch.Generator(device="cuda").manual_seed(4)
    chosen = torch.rand(tokens, 10, generator=g, device="cuda").argsort(1)[:, :top_k].int()
    chosen[::4, 3] = -1
    dw = torch.randn(tokens, top_k, generator=g, device="cuda")
    d = fg.moe_route_backward(l, of(chosen), dw)
    x, ok, at = l.double(), chosen >= 0, chosen.clamp(min=0).long()
    q = torch.softmax(torch.where(ok, torch.gather(x, 1, at), -INF), 1)
    w = torch.where(ok, dw.double(), 0.0)
    mean, size = (q * w).sum(1, keepdim=True), (q * w.abs()).sum(1, keepdim=True)
    want = torch.zeros_like(x).scatter_add_(1, at, q * (w - mean))
    mag = torch.zeros_like(x).scatter_add_(1, at, q * (w.abs() + size))
    assert (want.abs().amax(1) > 1e-3).sum() > tokens // 2
    ref.within(d, want, ref.REL * mag + EPS[dtype] * want.abs() + 1e-38)


def test_one_choice_of_infinity():
    l = logits_of(3, 8, 5)
    l[0, 1] = INF           # not chosen
    l[1, 2] = l[1, 3] = INF  # both chosen, with a finite one
    l[2, 4] = INF           # chosen, twice
    chosen = torch.tensor([[2, 3, 4], [2, 3, 4], [4, 5, 4]])
    dw = torch.tensor([[1.0, 2.0, 4.0]] * 3, device="cuda")
    d = fg.moe_route_backward(l, of(chosen), dw).double()
    assert torch.isfinite(d).all()
    q = torch.softmax(l[0, 2:5].double(), 0)
    want = q * (dw[0].double() - (q * dw[0].double()).sum())
    ref.within(d[0, 2:5], want, ref.REL * (q * 8))
    same(d[1], torch.tensor([0, 0, -0.25, 0.25, 0, 0, 0, 0], device="cuda", dtype=torch.float64))
    same(d[2], torch.zeros(8, device="cuda", dtype=torch.float64))
