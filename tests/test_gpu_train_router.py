"""The balance loss, its counts, and the gradient of the router's logits.

32-bit sums of probabilities, each off by at most 2^-20 of itself (two fast
functions and the softmax's sum): everything is held to REL = 2^-18 of the
magnitudes that are added, and half a step of the output's type.
"""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref
from tests.test_gpu_train_columns import INF, NAN, same

pytestmark = pytest.mark.gpu

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def logits_of(tokens, experts, seed, dtype=torch.float32, padded=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = 2 * torch.randn(tokens, experts, generator=g, device="cuda")
    l[torch.rand(tokens, generator=g, device="cuda") < padded] = -INF
    return l.to(dtype)


def softmax64(l):
    l = l.double()
    l = torch.where(torch.isnan(l), -INF, l)
    top = l.amax(1, keepdim=True)
    some = top > -INF
    p = torch.where(l == top, 1.0, torch.exp(l - torch.where(some, top, 0.0)))
    p = torch.where(some & (l > -INF), p, 0.0)
    return torch.where(some, p / p.sum(1, keepdim=True).clamp(min=1e-300), 0.0), some[:, 0]


def balance64(l, offsets, c):
    p, some = softmax64(l)
    e, n = l.shape[1], int(some.sum())
    counts = (offsets[1:] - offsets[:-1]).long().clamp(min=0)
    f = counts.double() / max(int(counts.sum()), 1)
    probs = p.sum(0) / n if n else torch.zeros(e, dtype=torch.float64, device="cuda")
    slopes = c * e * f / n if n else torch.zeros_like(f)
    return c * e * (f * probs).sum(), counts, probs, slopes


def backward64(l, experts, dw, slopes, renormalize):
    """Gradient and the magnitudes that its error is measured by."""
    p, _ = softmax64(l)
    d, mag = torch.zeros_like(p), torch.zeros_like(p)
    if slopes is not None:
        s = slopes.double()
        d += p * (s - (p * s).sum(1, keepdim=True))
        mag += p * (s.abs() + (p * s.abs()).sum(1, keepdim=True))
    if dw is not None:
        ok, at = experts >= 0, experts.clamp(min=0).long()
        q = torch.where(ok, torch.gather(p, 1, at), 0.0)
        w = torch.where(ok, dw.double(), 0.0)
        if renormalize:
            q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
            d.scatter_add_(1, at, q * (w - (q * w).sum(1, keepdim=True)))
            mag.scatter_add_(1, at, q * (w.abs() + (q * w.abs()).sum(1, keepdim=True)))
        else:
            d.scatter_add_(1, at, q * w)
            d -= p * (q * w).sum(1, keepdim=True)
            mag.scatter_add_(1, at, q * w.abs())
            mag += p * (q * w.abs()).sum(1, keepdim=True)
    return d, mag


SHAPES = [(1, 8, 2), (1, 1, 1), (3, 33, 4), (61, 64, 8), (64, 1024, 32), (65, 96, 6), (500, 7, 3), (3000, 256, 8), (2049, 384, 1),
          (700, 1000, 5)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,experts,top_k", SHAPES)
def test_balance_and_gradient(tokens, experts, top_k, dtype):
    l = logits_of(tokens, experts, 1, dtype, padded=0.1 if tokens > 3 else 0.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    dw = torch.randn(tokens, top_k, generator=g, device="cuda")
    for renormalize in (True, False):
        r = fg.moe_route(l, top_k, renormalize=renormalize)
        b = fg.moe_balance_loss(l, r.offsets, 0.25)
        loss, counts, probs, slopes = balance64(l, r.offsets, 0.25)
        assert b.loss.shape == () and abs(b.loss.item() - loss.item()) <= ref.REL * abs(loss.item())
        same(b.counts.long(), counts)
        ref.within(b.probs, probs, ref.REL * probs)
        ref.within(b.slopes, slopes, ref.REL * slopes)
        for w, s in ((dw, b.slopes), (dw, None), (None, b.slopes), (None, None)):
            d = fg.moe_route_backward(l, r, w, slopes=s, renormalize=renormalize)
            want, mag = backward64(l, r.experts, w, s, renormalize)
            assert d.dtype == dtype and d.shape == l.shape
            ref.within(d, want, ref.REL * mag + EPS[dtype] * want.abs() + 1e-38)


def test_rows_with_nothing_and_values_that_are_not_numbers():
    l = logits_of(40, 16, 3)
    l[0] = -INF
    l[1] = NAN
    l[2, :3] = INF
    l[3, 5] = NAN
    l[4, :15] = -INF
    l[5] = 3e38
    l[6] = -3e38
    r = fg.moe_route(l, 4)
    b = fg.moe_balance_loss(l, r.offsets, 1.0)
    loss, counts, probs, slopes = balance64(l, r.offsets, 1.0)
    same(b.counts.long(), counts)
    assert ((b.probs.double() - probs).abs() <= ref.REL * probs).all() and abs(b.loss.item() - loss.item()) <= ref.REL * loss.item()
    dw = torch.randn(40, 4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    for renormalize in (True, False):
        d = fg.moe_route_backward(l, r, dw, slopes=b.slopes, renormalize=renormalize)
        want, mag = backward64(l, r.experts, dw, b.slopes, renormalize)
        ref.within(d, want, ref.REL * mag + 2.0 ** -24 * want.abs())
        assert not d[:2].any()


def test_no_tokens_and_tokens_with_nothing():
    offsets = torch.zeros(9, dtype=torch.int32, device="cuda")
    for l in (torch.empty(0, 8, device="cuda"), torch.full((5, 8), -INF, device="cuda"), torch.full((300, 8), NAN, device="cuda")):
        b = fg.moe_balance_loss(l, offsets, 1.0)
        assert b.loss.item() == 0 and not b.counts.any() and not b.probs.any() and not b.slopes.any()
        assert not fg.moe_route_backward(l, (None, None), slopes=b.slopes).any()


def test_views_of_logits():
    """Rows of any distance and alignment."""
    for dtype in (torch.float32, torch.bfloat16):
        for at, step in ((0, 1), (1, 1), (3, 2)):
            big = logits_of(200, 150, 5, dtype)
            l = big[::step, at:at + 65]
            r = fg.moe_route(l, 3)
            c = l.contiguous()
            for x, y in zip(fg.moe_balance_loss(l, r.offsets), fg.moe_balance_loss(c, r.offsets)):
                same(x, y)
            dw = torch.ones(l.shape[0], 3, device="cuda").cumsum(1)
            same(fg.moe_route_backward(l, r, dw), fg.moe_route_backward(c, r, dw))


def test_the_same_bits_each_time():
    l = logits_of(5000, 128, 6)
    r = fg.moe_route(l, 8)
    first = fg.moe_balance_loss(l, r.offsets)
    for _ in range(3):
        for x, y in zip(first, fg.moe_balance_loss(l, r.offsets)):
            same(x, y)


def test_experts_out_of_range_are_no_choice():
    l = logits_of(4, 8, 7)
    experts = torch.tensor([[0, 8], [-1, 3], [1 << 30, -(1 << 31)], [2, 2]], dtype=torch.int32, device="cuda")
    dw = torch.ones(4, 2, device="cuda")
    d = fg.moe_route_backward(l, (None, experts), dw)
    assert torch.isfinite(d).all() and not d[2].any()
    same(d[0], torch.zeros(8, device="cuda"))       # one choice: its weight is 1 whatever the logits


@pytest.mark.parametrize("renormalize", [True, False])
def test_against_differences(renormalize):
    """Balance loss plus <weights, dw> of the fixed choice, by central differences in 64 bits."""
    l = logits_of(30, 12, 8)
    r = fg.moe_route(l, 3, renormalize=renormalize)
    dw = torch.randn(30, 3, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    b = fg.moe_balance_loss(l, r.offsets, 0.5)
    d = fg.moe_route_backward(l, r, dw, slopes=b.slopes, renormalize=renormalize).double()
    h = 1e-5

    def value(x):
        p = torch.softmax(x, 1)
        q = torch.gather(p, 1, r.experts.long())
        q = q / q.sum(1, keepdim=True) if renormalize else q
        f = (r.offsets[1:] - r.offsets[:-1]).double() / int(r.offsets[-1])
        return 0.5 * 12 * (f * p.mean(0)).sum() + (q * dw.double()).sum()

    x = l.double()
    for t in range(0, 30, 7):
        for e in range(12):
            step = torch.zeros_like(x)
            step[t, e] = h
            num = (value(x + step) - value(x - step)) / (2 * h)
            # h^2 of third derivatives below 10 |dw|, rounding of sums below 100 at 1e-16 / h, and REL of the terms
            assert abs(d[t, e] - num) <= 10 * h * h * 3 + 1e-9 + ref.REL * 6 * dw.abs().max()


def test_refusals():
    l = logits_of(10, 8, 10)
    r = fg.moe_route(l, 2)
    dw = torch.zeros(10, 2, device="cuda")
    for call, match in [
            (lambda: fg.moe_balance_loss(l, r.offsets[:8].contiguous()), "offsets"),
            (lambda: fg.moe_balance_loss(l, r.offsets.long()), "dtype"),
            (lambda: fg.moe_balance_loss(l.half(), r.offsets), "dtype"),
            (lambda: fg.moe_balance_loss(l, r.offsets, "much"), "coefficient"),
            (lambda: fg.moe_route_backward(l, r, dw[:9].contiguous()), "dweights"),
            (lambda: fg.moe_route_backward(l, r, dw.double()), "dtype"),
            (lambda: fg.moe_route_backward(l, r, slopes=torch.zeros(9, device="cuda")), "slopes"),
            (lambda: fg.moe_route_backward(l, (None, None), dw), "dweights")]:
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(fg.FgError, match="experts"):
        x = logits_of(4, 1100, 11)
        fg.moe_balance_loss(x, torch.zeros(1101, dtype=torch.int32, device="cuda"))
