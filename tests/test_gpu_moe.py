"""Routing and the weighted sum of the experts' rows against plain
implementations in 64 bits.

Routing's order is compared for equality.  A weight is exp() of a difference
(the difference rounded once, expf 2 ulp) over a sum of at most E such terms
and one division: (8 + |l - top|) * 2^-23 relative, E < 2^7 additions' worth more
when all experts are summed.  The weighted sum: top_k + 1 fused 32-bit steps and
one rounding to bf16.
"""
import numpy as np
import pytest
import torch

import mx_gemm_gb300 as fg

pytestmark = pytest.mark.gpu


def route_reference(logits, k, renormalize):
    l = logits.double().cpu().numpy()
    l = np.where(np.isnan(l), -np.inf, l) + 0.0
    t, e = l.shape
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    v = np.take_along_axis(l, order, axis=1)
    ok = v > -np.inf
    top = v[:, :1]
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.where(ok, np.exp(np.where(v == top, 0.0, v - top)), 0.0)
        every = np.where(l > -np.inf, np.exp(np.where(l == top, 0.0, l - top)), 0.0)
    total = (p if renormalize else every).sum(axis=1, keepdims=True)
    w = np.divide(p, total, out=np.zeros_like(p), where=ok)
    experts = np.where(ok, order, -1)
    flat = np.where(ok, order, e).reshape(-1)
    perm = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[perm], np.arange(e + 1))
    rows = np.where(flat[perm] < e, perm // k, -1)
    slots = np.empty(t * k, np.int64)
    slots[perm] = np.arange(t * k)
    return w, experts, offsets, rows, np.where(ok, slots.reshape(t, k), -1)


def check_route(logits, k, renormalize=True):
    got = fg.moe_route(logits, k, renormalize=renormalize)
    want = route_reference(logits, k, renormalize)
    for name, g, w in list(zip(got._fields, got, want))[1:]:
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w), name
    w = got.weights.double().cpu().numpy()
    assert (np.abs(w - want[0]) <= 160 * 2.0 ** -23 * want[0] + 1e-37).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 2), (1, 128, 8), (2, 33, 5), (31, 60, 4), (63, 64, 8), (64, 256, 8),
                                   (65, 256, 8), (129, 40, 40 - 8), (777, 160, 6), (4099, 512, 8), (10000, 1000, 3),
                                   (16384, 256, 8), (40000, 7, 1)])
def test_route(dtype, t, e, k):
    g = torch.Generator(device="cuda").manual_seed(t + e)
    logits = (3 * torch.randn(t, e, generator=g, device="cuda") + torch.randn(e, generator=g, device="cuda")).to(dtype)
    check_route(logits, k)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("t", [40, 300])
def test_route_masked_equal_and_not_finite_logits(renormalize, t):
    g = torch.Generator(device="cuda").manual_seed(t)
    logits = torch.randn(t, 48, generator=g, device="cuda").round()     # many ties
    logits[3] = -float("inf")                                           # a padding token
    logits[4] = 0.0
    logits[5, 1::2] = -0.0                                              # both zeros are equal
    logits[5, 0::2] = 0.0
    logits[6, 2:] = -float("inf")                                       # fewer than top_k
    logits[7] = torch.finfo(torch.float32).min                          # the type's lowest value is a logit
    logits[8, 10:] = torch.finfo(torch.float32).min
    logits[9, 7] = float("nan")
    logits[10] = float("nan")
    logits[11, 30] = float("inf")
    logits[12, [5, 20]] = float("inf")
    logits[13] = -1e-45
    logits[20:30] = -float("inf")
    check_route(logits, 6, renormalize)


def test_route_all_padding_and_no_tokens():
    for t in (5, 200):
        r = fg.moe_route(torch.full((t, 32), -float("inf"), device="cuda"), 4)
        assert (r.weights == 0).all() and (r.offsets == 0).all()
        assert all((x == -1).all() for x in (r.experts, r.rows, r.slots))
    r = fg.moe_route(torch.empty(0, 32, device="cuda"), 4)
    assert (r.offsets == 0).all() and r.rows.numel() == 0


def test_route_row_distance_and_odd_start():
    g = torch.Generator(device="cuda").manual_seed(8)
    wide = torch.randn(100, 300, generator=g, device="cuda").to(torch.bfloat16)
    check_route(wide[:, 3:3 + 97], 5)
    check_route(wide[7:8, 1:100], 5)


def combine_reference(y, slots, weights, residual):
    out = residual.double() if residual is not None else torch.zeros(slots.shape[0], y.shape[1], dtype=torch.float64, device=y.device)
    size = out.abs()
    for j in range(slots.shape[1]):
        s = slots[:, j].long()
        ok = (s >= 0) & (s < y.shape[0])
        term = torch.where(ok, weights[:, j].double(), 0.0)[:, None] * torch.where(ok[:, None], y[s.clamp(0, y.shape[0] - 1)].double(), 0.0)
        out = out + term
        size = size + term.abs()
    return out, size


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("t,k,n", [(1, 8, 7168), (1, 1, 8), (5, 2, 1000), (77, 9, 1032), (300, 8, 2048), (3, 32, 512)])
def test_combine(t, k, n, residual):
    g = torch.Generator(device="cuda").manual_seed(t * n + k)
    y = torch.randn(t * k, n, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(t * k, generator=g, device="cuda").view(t, k).int()
    weights = torch.rand(t, k, generator=g, device="cuda")
    if t > 4:
        slots[2] = -1            # a padding token: the residual alone
        slots[3, -1] = -1
        slots[4, 0] = t * k      # out of range is no choice
        y[int(slots[0, 0])] = float("nan")
        y[int(slots[1, 0]), 0] = float("inf")
    r = torch.randn(t, n, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    out = fg.moe_combine(y, slots, weights, residual=r)
    want, size = combine_reference(y, slots, weights, r)
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isinf(out), torch.isinf(want))
    bound = 2.0 ** -8 * want.abs() + (k + 1) * 2.0 ** -23 * size
    assert ((out.double() - want).abs() <= bound)[finite].all()


def test_combine_nan_rows_of_dropped_choices_stay_out():
    """A dropped choice (slot -1) contributes nothing, whatever its weight holds."""
    y = torch.full((2, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    slots = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    weights = torch.full((3, 2), float("nan"), device="cuda")
    assert (fg.moe_combine(y, slots, weights) == 0).all()


def test_combine_past_32_bits_of_elements():
    """Rows of Y beyond element 2^31: the first and last tokens against the formula."""
    n, r = 8192, 270_000                    # 2.2e9 elements
    y = torch.empty(r, n, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    edge = torch.randn(64, n, generator=g, device="cuda").to(torch.bfloat16)
    y[:32], y[-32:] = edge[:32], edge[32:]
    slots = torch.cat([torch.arange(32), torch.arange(r - 32, r)]).int().cuda().view(32, 2)
    weights = torch.rand(32, 2, generator=g, device="cuda")
    want, size = combine_reference(edge, torch.arange(64, device="cuda").int().view(32, 2), weights, None)
    assert ((fg.moe_combine(y, slots, weights).double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all()


@pytest.mark.parametrize("call,text", [
    (lambda x, i: fg.moe_route(x, 0), "top_k"),
    (lambda x, i: fg.moe_route(x, 9), "top_k"),
    (lambda x, i: fg.moe_route(x.t(), 2), "contiguous rows"),
    (lambda x, i: fg.moe_route(x.double(), 2), "dtype"),
    (lambda x, i: fg.moe_route(x[0], 2), "2-D"),
    (lambda x, i: fg.moe_route(x.expand(4, 8)[:, :1].expand(4, 8), 2), "rows"),
    (lambda x, i: fg.moe_combine(x, i, x), "dtype"),
    (lambda x, i: fg.moe_combine(x.to(torch.bfloat16), x, x), "dtype"),
    (lambda x, i: fg.moe_combine(x.to(torch.bfloat16), i, x[:, :3].contiguous()), "shape"),
    (lambda x, i: fg.moe_combine(x.to(torch.bfloat16), i.t(), x), "contiguous"),
    (lambda x, i: fg.moe_combine(x.to(torch.bfloat16), i, x, residual=x.to(torch.bfloat16)[:2]), "residual"),
])
def test_binding_refusals(call, text):
    x = torch.zeros(4, 8, device="cuda")
    i = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match=text):
        call(x, i)


def test_library_refusals_come_as_errors():
    with pytest.raises(fg.FgError) as e:
        fg.moe_route(torch.zeros(2, 2000, device="cuda"), 2)      # more experts than it takes
    assert e.value.status == fg.FG_ERR_SHAPE and "1024" in str(e.value)
    with pytest.raises(fg.FgError) as e:
        fg.moe_combine(torch.zeros(2, 12, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, device="cuda"))
    assert e.value.status == fg.FG_ERR_SHAPE
