"""The training step of examples/moe_training.py: its gradients against those of the
layer in 64 bits (the same routing and the unquantised weights), a captured step, and
the calls on other streams, devices' other memory, and from several threads.

Bound of a gradient.  An e4m3 code is off by up to 2^-4 of its value, 2^-4 / sqrt(3) =
3.6 % in the mean square at most; sums keep that relative size.  Between the inputs
and the weights' or the input's gradient lie at most eight such roundings (tokens,
their columns, gate / up weights, checkpoint, output gradient, down weights, activation
gradient, its columns), the gate's own twice: sqrt(9) * 3.6 % = 11 %.  Bound: twice.
The routing weights' gradients pass five: 8 %; bound 16 %, of the logits' gradient too.
"""
import threading

import pytest
import torch

import mx_gemm_gb300 as fg
from examples import moe_training
from tests import train_ref as ref
from tests.test_gpu_streams import SLOW, raw, same

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 384, 12, 3


def make(mode, tokens, seed=1, padded=False):
    layer = moe_training.random_layer(mode, H, I, E, K, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, dy = (torch.randn(tokens, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    if padded:
        x[::7] = 0
    return layer, x, dy


def gradients64(layer, x, dy, kept):
    """Gradients of sum(dy * output) + balance loss at the kept routing, by autograd in 64 bits."""
    leaves = [t.double().detach().requires_grad_() for t in (x, layer.router, layer.gate_up, layer.down)]
    x, router, gate_up, down = leaves
    logits = x @ router.T
    chosen = kept.routing.experts.long()
    weights = torch.softmax(torch.gather(logits, 1, chosen), dim=1)
    out = torch.zeros_like(x)
    for e in range(E):
        t, j = (chosen == e).nonzero(as_tuple=True)
        if t.numel():
            g, u = (x[t] @ gate_up[e].T).chunk(2, dim=1)
            out = out.index_add(0, t, weights[t, j][:, None] * ((g * torch.sigmoid(g) * u) @ down[e].T))
    f = (kept.routing.offsets[1:] - kept.routing.offsets[:-1]).double() / int(kept.routing.offsets[-1])
    balance = layer.balance * E * (f * torch.softmax(logits, dim=1).mean(0)).sum()
    return out.detach(), balance.detach(), torch.autograd.grad((out * dy.double()).sum() + balance, leaves)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("mode", ref.MODES)
@pytest.mark.parametrize("tokens", [1, 50, 700, 3000])
def test_gradients(mode, tokens):
    layer, x, dy = make(mode, tokens)
    y, kept = layer.forward(x)
    got = layer.backward(dy, kept)
    out, balance, want = gradients64(layer, x, dy, kept)
    assert off(y, out) <= 0.16 and abs(float(kept.balance.loss) - float(balance)) <= 1e-5 * float(balance)
    for name, g, w in zip(got._fields, got, want):
        assert off(g, w) <= (0.16 if name == "router" else 0.22), name
    routed = torch.zeros(E, dtype=torch.bool, device="cuda")
    routed[kept.routing.experts.flatten().long()] = True
    assert not got.gate_up[~routed].any() and not got.down[~routed].any()
    assert fg.get_error() == fg.FG_OK


@pytest.mark.parametrize("mode", ref.MODES)
def test_a_captured_step_gives_the_same_bits(mode):
    for tokens in (3, 900):
        layer, x, dy = make(mode, tokens, seed=3)

        def step():
            y, kept = layer.forward(x)
            return (y, kept.balance.loss.view(1), *layer.backward(dy, kept))

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for seed in (4, 5):
            for t, s in zip((x, dy), make(mode, tokens, seed)[1:]):
                t.copy_(s)
            for t in out:
                t.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            assert same(got, step())


def test_two_steps_at_once():
    """Two streams, each with a step of its own, with nothing between them."""
    jobs = [make("fp8_block128", 600, 6), make("mxfp8_b32", 900, 8)]

    def step(layer, x, dy):
        y, kept = layer.forward(x)
        return (y, kept.balance.loss.view(1), *layer.backward(dy, kept))

    want = [step(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [None, None]
    errors = []

    def run(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(5):
                    got[i] = step(*jobs[i])
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and all(same(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------- another stream

def rows(seed, m, k):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)


def weight(seed):
    w = rows(seed, 2048, 4096).view(4, 512, 4096)
    return lambda **kw: fg.quantize_weight("fp8_block128", w, transpose=True, **kw)


def checkpoint(seed):
    x = rows(seed, 2000, 4096)
    return lambda **kw: fg.swiglu_checkpoint("mxfp8_b32", x, **kw)


def columns(seed):
    x = rows(seed, 3000, 1024)
    r, _ = ref.routing(1000, 16, 3, seed)

    def call(**kw):
        c = fg.quantize_columns(x, r.offsets, **kw)
        return c.data, c.sf
    return call


def swiglu(seed):
    r, _ = ref.routing(1000, 16, 3, seed)
    saved, scales = fg.quantize("mxfp8", rows(seed, 3000, 2048))
    dy = rows(seed + 1, 3000, 1024)

    def call(**kw):
        d = fg.swiglu_backward("mxfp8", dy, saved, scales, routing=r, columns=True, plain=True, **kw)
        return (d.codes, d.scales, d.dx, d.dweights, d.dx_columns.data, d.dx_columns.sf, d.act_columns.data, d.act_columns.sf)
    return call


def wgrad(seed):
    r, _ = ref.routing(1000, 16, 3, seed)
    a, b = fg.quantize_columns(rows(seed, 3000, 512), r.offsets), fg.quantize_columns(rows(seed + 1, 3000, 1024), r.offsets)
    return lambda **kw: (fg.grouped_wgrad(a, b, r.offsets, **kw),)


def balance(seed):
    l = rows(seed, 5000, 256)
    r = fg.moe_route(l, 8)
    return lambda **kw: tuple(t.view(-1) for t in fg.moe_balance_loss(l, r.offsets, 1.0, **kw))


def route_backward(seed):
    l = rows(seed, 5000, 256)
    r = fg.moe_route(l, 8)
    dw = rows(seed + 1, 5000, 8).float()
    return lambda **kw: (fg.moe_route_backward(l, r, dw, **kw),)


CALLS = {f.__name__: f for f in (weight, checkpoint, columns, swiglu, wgrad, balance, route_backward)}


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_memory_that_the_current_stream_still_uses(name, handle):
    """Blocks of the outputs' and the workspaces' sizes are freed with slow writes to them pending on the current
    stream; the call's stream does not wait for those, so the call must not be given the blocks."""
    call = CALLS[name](1)
    want = call()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty_like(t) for t in raw(want) for _ in range(3)]
    blocks += [torch.empty(1 << s, dtype=torch.uint8, device="cuda") for s in range(9, 27) for _ in range(2)]
    blocks[0].fill_(0)
    torch.cuda.synchronize()
    torch.cuda._sleep(SLOW)
    for b in blocks:
        b.fill_(0xff)
    del blocks, b
    got = call(stream=other.cuda_stream if handle else other)
    assert not torch.cuda.current_stream().query()    # the writes are still to come
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_that_the_current_stream_still_reads(name):
    first, second = CALLS[name](1), CALLS[name](2)
    want = first()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = first(stream=other)
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(SLOW)
    copies = [t.clone() for t in raw(got)]
    del got
    later = [second(stream=other) for _ in range(4)]
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, raw(want))) and same(later[0], later[3])


@pytest.mark.parametrize("name", list(CALLS))
def test_a_captured_call_replays(name):
    call = CALLS[name](3)
    want = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        for t in raw(out):
            t.fill_(0x5a)
        graph.replay()
        assert same(out, want)
    assert fg.get_error() == fg.FG_OK
