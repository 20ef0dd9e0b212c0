"""The mixture-of-experts layer of examples/moe_layer.py end to end.

Against the layer in 64 bits on the same (quantised) weights with unquantised
activations and the layer's own routing.  An e4m3 code is off by up to 2^-4 of
its value, 2.6 % in the mean square; the sums keep that relative size, the
product of gate and up adds two such errors (silu' up to 1.1) and is rounded
again: about 2.6 % * sqrt(2 * 1.1 + 1) = 4.7 %.  Bound: 8 %.  For 4-bit
activations (e2m1: 2^-2, about 11 %) the same gives 20 %; bound 30 %.
"""
import pytest
import torch

import mx_gemm_gb300 as fg
from examples import moe_layer
from tests.test_gpu_grouped import values

pytestmark = pytest.mark.gpu

H, I, E, K = 1024, 512, 24, 4


def make(mode):
    layer, w = moe_layer.random_layer(mode, H, I, E, K, seed=3)
    wmode = "mxfp4" if mode == "mxfp4_fp8a" else mode
    exact = {n: values(*fg.quantize(wmode, w[n].flatten(0, 1)), wmode).view(w[n].shape) for n in ("gate_up", "down")}
    return layer, w, exact


def reference(w, exact, x, residual, routing, eps=1e-6):
    """The experts' contribution, fp64 [T][H]."""
    h = x.double() + residual.double()
    y = h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + eps) * w["norm"].to(torch.bfloat16).double()
    out = torch.zeros_like(h)
    for j in range(K):
        for e in range(E):
            t = (routing.experts[:, j] == e).nonzero()[:, 0]
            if t.numel():
                g, u = (y[t] @ exact["gate_up"][e].T).chunk(2, dim=1)
                out[t] += routing.weights[t, j].double()[:, None] * ((g * torch.sigmoid(g) * u) @ exact["down"][e].T)
    return h, out


@pytest.mark.parametrize("mode", ["mxfp8_b32", "mxfp8", "mxfp4_fp8a", "mxfp4"])
@pytest.mark.parametrize("tokens", [1, 7, 100, 1500])
def test_layer(mode, tokens):
    layer, w, exact = make(mode)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, residual = (torch.randn(tokens, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, routing = layer(x, residual)
    h, want = reference(w, exact, x, residual, routing)
    err = (out.double() - h - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()
    # out is h + contribution rounded to bf16: that rounding is of the sum
    rounding = 2.0 ** -9 * (h + want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()
    assert err <= (0.30 if mode == "mxfp4" else 0.08) + 2 * rounding, (float(err), float(rounding))
    assert fg.get_error() == fg.FG_OK


def test_layer_in_a_graph_gives_the_same_bits():
    layer, _, _ = make("mxfp8_b32")
    for tokens in (1, 300):
        x, residual = (torch.randn(tokens, H, device="cuda").to(torch.bfloat16) for _ in range(2))
        want, _ = layer(x, residual)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, _ = layer(x, residual)
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)


def test_tokens_do_not_depend_on_one_another():
    """A NaN token leaves the others' bits alone, and its own output is NaN."""
    layer, _, _ = make("mxfp8_b32")
    x, residual = (torch.randn(50, H, device="cuda").to(torch.bfloat16) for _ in range(2))
    want, r0 = layer(x, residual)
    x[7, 100] = float("nan")
    out, r = layer(x, residual)
    keep = torch.arange(50, device="cuda") != 7
    assert torch.isnan(out[7]).any() and (r.experts[7] == -1).all()
    assert torch.equal(r.experts[keep], r0.experts[keep]) and torch.equal(out[keep], want[keep])
