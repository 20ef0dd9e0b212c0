"""Calls on another stream than the current one, without more waits than the
caller's tensors need: memory that the call allocates must not be in use on the
current stream, and what the caller lets go of must not be reused too early."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests.test_gpu_grouped import Experts

pytestmark = pytest.mark.gpu

SLOW = 100_000_000  # clock cycles: 50 ms, while a call takes under one


def quantize(seed):
    x = rows(seed, 2000, 4096)
    return lambda **kw: fg.quantize("mxfp8_b32", x, act="swiglu", **kw)


def norm(seed):
    x, r, w = rows(seed, 2000, 2048), rows(seed + 10, 2000, 2048), rows(seed + 20, 1, 2048)[0]
    return lambda **kw: fg.rmsnorm_quantize("mxfp4", x, w, residual=r, normed=True, **kw)


def route(seed):
    x = rows(seed, 5000, 256)
    return lambda **kw: tuple(fg.moe_route(x, 8, **kw))


def grouped(total):
    def make(seed):
        c = Experts("mxfp8_b32", [total // 8] * 8, 1024, 4096, seed, gather_from=100)
        return lambda **kw: (c.run(**kw),)
    return make


def combine(seed):
    y = rows(seed, 8000, 1024)
    g = torch.Generator(device="cuda").manual_seed(seed)
    slots = torch.randperm(8000, generator=g, device="cuda").view(2000, 4).int()
    weights = torch.rand(2000, 4, generator=g, device="cuda")
    return lambda **kw: (fg.moe_combine(y, slots, weights, **kw),)


def rows(seed, m, k):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)


class Dense:
    """Preshuffling, product, two-pass product and inverse on one weight, each on the stream that it is given."""

    def __init__(self, mode, m, n, k, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.mode, self.m, self.n, self.k = mode, m, n, k
        self.a, self.a_s = fg.quantize(mode, torch.randn(m, k, generator=g, device="cuda"))
        self.b, self.b_s = fg.quantize(mode, torch.randn(n, k, generator=g, device="cuda"))
        self.pb = fg.preshuffle_b(mode, self.b, self.b_s)
        self.partials = torch.randn(4 * m * n, generator=g, device="cuda")

    def gemm(self, split_k, **kw):
        return (fg.gemm(self.a, self.pb, self.a_s, split_k=split_k, **kw),)

    def preshuffle(self, **kw):
        pb = fg.preshuffle_b(self.mode, self.b, self.b_s, **kw)
        return pb.data, pb.sf

    def unshuffle(self, **kw):
        return fg.unshuffle_b(self.pb, **kw)

    def reduce(self, **kw):
        return (fg.gemm_splitk_reduce(self.partials, 4, self.m, self.n, **kw),)


def dense(m, call, split_k=None):
    def make(seed):
        d = Dense("mxfp8_b32", m, 2048, 7168, seed)
        return (lambda **kw: d.gemm(split_k, **kw)) if call == "gemm" else getattr(d, call)
    return make


CALLS = {"quantize": quantize, "norm": norm, "route": route, "grouped_few": grouped(24), "grouped_many": grouped(4096),
         "combine": combine, "gemm_one": dense(1, "gemm", 0), "gemm_two_pass": dense(16, "gemm", 16),
         "gemm_many": dense(1000, "gemm", 0), "preshuffle": dense(16, "preshuffle"), "unshuffle": dense(16, "unshuffle"),
         "reduce": dense(16, "reduce")}


def raw(ts):
    return [t.contiguous().view(torch.uint8) for t in ts if t is not None]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(raw(a), raw(b)))


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_memory_that_the_current_stream_still_uses(name, handle):
    """Blocks of the outputs' and the workspaces' sizes are freed with slow writes to them pending on the current
    stream.  The call's stream does not wait for that stream, so the call must not be given those blocks."""
    call = CALLS[name](1)
    want = call()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty_like(t) for t in raw(want) for _ in range(3)]
    blocks += [torch.empty(1 << s, dtype=torch.uint8, device="cuda") for s in range(9, 27) for _ in range(2)]
    blocks[0].fill_(0)  # a kernel's first launch, which loads it, waits for the device
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
    """Outputs freed while the current stream has yet to read them are not overwritten by the next call."""
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


def test_inputs_let_go_while_the_stream_still_reads_them():
    x = rows(3, 2000, 4096)
    want = fg.quantize("mxfp8_b32", x)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(SLOW)
    twin = x.clone()
    torch.cuda.current_stream().synchronize()
    got = fg.quantize("mxfp8_b32", twin, stream=other)
    del twin
    junk = [torch.full_like(x, 7.0) for _ in range(4)]
    assert not other.query() and len(junk) == 4
    torch.cuda.synchronize()
    assert same(got, want)


def test_default_stream_by_its_handles():
    x = rows(4, 300, 1024)
    want = fg.quantize("mxfp8_b32", x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for handle in (0, 1):
            got = fg.quantize("mxfp8_b32", x, stream=handle)
            torch.cuda.synchronize()
            assert same(got, want)
