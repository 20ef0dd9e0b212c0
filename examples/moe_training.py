"""A training step of a mixture-of-experts feed-forward layer in 8 bits.

    python examples/moe_training.py [--mode fp8_block128] [--tokens 4096]

Forward: the tokens in 8 bits, routing with its balance loss, the gate / up products
grouped by expert, the gated activation with its 8-bit checkpoint, the down products
and the weighted sum.  Kept for the backward pass: the tokens' codes and scales, the
checkpoint, the routing and the router's logits.  Backward: the down products' input
gradients (the output's gradient quantised once a token and gathered), the
activation's backward pass, which leaves its gradients in both 8-bit forms, the
weights' gradients, the input's, and the logits'.

The weights are kept in fp32 and quantised and laid out, as they are and transposed, by
update(), which follows every change of theirs: it is timed by itself, beside the steps.
Nothing waits for the device, so a step can be captured in a CUDA graph.
"""
import argparse
import os
import sys
from typing import NamedTuple

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mx_gemm_gb300 as fg  # noqa: E402


class Kept(NamedTuple):
    """What the forward pass leaves for the backward pass."""
    codes: torch.Tensor         # the tokens, e4m3 [T][H]
    scales: torch.Tensor
    x: torch.Tensor             # ... and as they came, for the router's weight
    logits: torch.Tensor
    routing: fg.Routing
    balance: fg.Balance
    saved: torch.Tensor         # the checkpoint of gate and up
    saved_scales: torch.Tensor


class Gradients(NamedTuple):
    x: torch.Tensor         # bf16 [T][H]
    router: torch.Tensor    # fp32 [E][H]
    gate_up: torch.Tensor   # fp32 [E][2 I][H]
    down: torch.Tensor      # fp32 [E][H][I]


class MoeTrainingLayer:
    """Weights in fp32: router [E][H]; gate_up [E][2 I][H] (gate rows, then up rows);
    down [E][H][I].  mode: an 8-bit block mode; H and I multiples of 128."""

    def __init__(self, mode, router, gate_up, down, top_k, balance=0.01):
        self.mode, self.top_k, self.balance = mode, top_k, balance
        self.router, self.gate_up, self.down = router, gate_up, down
        self.up, self.up_t = self._pair(gate_up)
        self.out, self.out_t = self._pair(down)

    def _pair(self, w):
        """Preshuffled weight [E * N][K] and its transpose [E * K][N]."""
        if self.mode == "fp8_block128":
            parts = [fg.quantize_weight(self.mode, w, transpose=t) for t in (False, True)]
        else:
            parts = [fg.quantize(self.mode, v.flatten(0, 1)) for v in (w, w.transpose(1, 2).contiguous())]
        return [fg.preshuffle_b(self.mode, *p) for p in parts]

    def update(self):
        """The 8-bit weights anew from the fp32 ones, in the memory that they have: a captured step reads them there."""
        for kept, w in (((self.up, self.up_t), self.gate_up), ((self.out, self.out_t), self.down)):
            for old, new in zip(kept, self._pair(w)):
                old.data.copy_(new.data)
                old.sf.copy_(new.sf)

    def forward(self, x):
        """(output bf16 [T][H], what backward() takes) of x bf16 [T][H]."""
        codes, scales = fg.quantize(self.mode, x)
        logits = x.float() @ self.router.T
        r = fg.moe_route(logits, self.top_k)
        balance = fg.moe_balance_loss(logits, r.offsets, self.balance)
        up = fg.grouped_gemm(codes, self.up, r.offsets, scales, rows=r.rows)
        act, act_scales, saved, saved_scales = fg.swiglu_checkpoint(self.mode, up)
        y = fg.grouped_gemm(act, self.out, r.offsets, act_scales)
        return fg.moe_combine(y, r.slots, r.weights), Kept(codes, scales, x, logits, r, balance, saved, saved_scales)

    def backward(self, dy, kept):
        """Gradients of <output, dy> + the balance loss."""
        r = kept.routing
        codes, scales = fg.quantize(self.mode, dy)
        dact = fg.grouped_gemm(codes, self.out_t, r.offsets, scales, rows=r.rows)
        d = fg.swiglu_backward(self.mode, dact, kept.saved, kept.saved_scales, routing=r, columns=True)
        dy_columns = fg.quantize_columns(dy, r.offsets, rows=r.rows)
        x_columns = fg.quantize_columns(kept.codes, r.offsets, scales=kept.scales, rows=r.rows)
        down = fg.grouped_wgrad(dy_columns, d.act_columns, r.offsets)
        gate_up = fg.grouped_wgrad(d.dx_columns, x_columns, r.offsets)
        dx = fg.grouped_gemm(d.codes, self.up_t, r.offsets, d.scales)
        dlogits = fg.moe_route_backward(kept.logits, r, d.dweights, slopes=kept.balance.slopes)
        from_router = (dlogits @ self.router).to(torch.bfloat16)
        dx = fg.moe_combine(dx, r.slots, torch.ones_like(r.weights), residual=from_router)
        return Gradients(dx, dlogits.T @ kept.x.float(), gate_up, down)


def random_layer(mode, hidden, inner, experts, top_k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return MoeTrainingLayer(mode, normal(experts, hidden) / hidden ** 0.5, normal(experts, 2 * inner, hidden) / hidden ** 0.5,
                            normal(experts, hidden, inner) / inner ** 0.5, top_k)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--mode", default="fp8_block128", choices=("fp8_block128", "mxfp8_b32", "mxfp8"))
    ap.add_argument("--tokens", type=int, nargs="+", default=[1024, 4096])
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=4)
    a = ap.parse_args()
    layer = random_layer(a.mode, a.hidden, a.inner, a.experts, a.top_k)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for n in (3, 10):
        start.record()
        for _ in range(n):
            layer.update()
        end.record()
    torch.cuda.synchronize()
    print("%s, %d experts, %d -> %d: the 8-bit weights anew %9.1f us" %
          (a.mode, a.experts, a.hidden, a.inner, start.elapsed_time(end) * 1000 / 10))
    for t in a.tokens:
        x, dy = (torch.randn(t, a.hidden, device="cuda").to(torch.bfloat16) for _ in range(2))

        def step():
            y, kept = layer.forward(x)
            return y, kept.balance.loss, layer.backward(dy, kept)

        for _ in range(3):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        start.record()
        for _ in range(10):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print("%s, %d experts, top %d, %d -> %d: %6d tokens %9.1f us a step, without that" %
              (a.mode, a.experts, a.top_k, a.hidden, a.inner, t, start.elapsed_time(end) * 1000 / 10))
    assert fg.get_error() == fg.FG_OK


if __name__ == "__main__":
    main()
