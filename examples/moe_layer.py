"""A mixture-of-experts feed-forward layer on preshuffled MX weights.

    python examples/moe_layer.py [--mode mxfp8_b32] [--tokens 1 64 4096]

One forward pass is seven calls: RMS norm with the residual's addition and
quantised output, the router's product, routing, the gate / up products grouped
by expert (rows gathered by token), the gated activation on its way to the A
format, the down products, and the weighted sum with the residual.  Nothing
waits for the device, so a pass can be captured in a CUDA graph.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mx_gemm_gb300 as fg  # noqa: E402


def _weight(mode, w):
    """Preshuffled weight of fp32 / bf16 w [N][K] in an MX mode."""
    return fg.preshuffle_b(mode, *fg.quantize("mxfp4" if mode == "mxfp4_fp8a" else mode, w))


class MoeLayer:
    """Weights: norm [H]; router [E][H]; gate_up [E][2 I][H] (gate rows, then up
    rows); down [E][H][I].  mode: an MX mode of the library."""

    def __init__(self, mode, norm, router, gate_up, down, top_k, eps=1e-6):
        self.mode, self.top_k, self.eps = mode, top_k, eps
        self.experts = router.shape[0]
        self.norm = norm.to(torch.bfloat16)
        rows = -self.experts % 128  # the GEMM takes N in tiles of 128
        self.router = fg.preshuffle_b("bf16", torch.nn.functional.pad(router.to(torch.bfloat16), (0, 0, 0, rows)))
        self.gate_up = _weight(mode, gate_up.flatten(0, 1))
        self.down = _weight(mode, down.flatten(0, 1))

    def __call__(self, x, residual):
        """(layer output added to the stream, bf16 [T][H]; the routing) of x, residual: bf16 [T][H]."""
        codes, scales, h, y = fg.rmsnorm_quantize(self.mode, x, self.norm, residual=residual, eps=self.eps, normed=True)
        logits = fg.gemm(y, self.router)
        r = fg.moe_route(logits[:, :self.experts], self.top_k)
        up = fg.grouped_gemm(codes, self.gate_up, r.offsets, scales, rows=r.rows)
        act, act_scales = fg.quantize(self.mode, up, act="swiglu")
        out = fg.grouped_gemm(act, self.down, r.offsets, act_scales)
        return fg.moe_combine(out, r.slots, r.weights, residual=h), r


def random_layer(mode, hidden, inner, experts, top_k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    gate_up = torch.stack([normal(2 * inner, hidden).to(torch.bfloat16) for _ in range(experts)]) / hidden ** 0.5
    down = torch.stack([normal(hidden, inner).to(torch.bfloat16) for _ in range(experts)]) / inner ** 0.5
    weights = dict(norm=1 + 0.1 * normal(hidden), router=normal(experts, hidden) / hidden ** 0.5, gate_up=gate_up, down=down)
    return MoeLayer(mode, top_k=top_k, **weights), weights


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--mode", default="mxfp8_b32", choices=("mxfp8_b32", "mxfp8", "mxfp4", "mxfp4_fp8a"))
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 64, 4096])
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    a = ap.parse_args()
    layer, _ = random_layer(a.mode, a.hidden, a.inner, a.experts, a.top_k)
    for t in a.tokens:
        x, residual = (torch.randn(t, a.hidden, device="cuda").to(torch.bfloat16) for _ in range(2))
        for _ in range(3):
            layer(x, residual)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(x, residual)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print("%s, %d experts, top %d, %d -> %d: %6d tokens %9.1f us a pass" %
              (a.mode, a.experts, a.top_k, a.hidden, a.inner, t, start.elapsed_time(end) * 1000 / 20))
    assert fg.get_error() == fg.FG_OK


if __name__ == "__main__":
    main()
