"""The training operators where indexes pass 32 bits: the last rows, experts and
columns of a large call against a small call on them alone, bit for bit."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref

pytestmark = pytest.mark.gpu

WIDE = 1 << 32


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 60 GB")
    yield
    torch.cuda.empty_cache()


def rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def same(a, b):
    assert a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def zeros(rows, cols, tail):
    """bf16 [rows][cols], zeros but for the last rows, which are `tail`."""
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-tail.shape[0]:] = tail
    return x


def test_weight():
    w = torch.zeros(11, 20480, 20480, dtype=torch.bfloat16, device="cuda")
    assert w.numel() > WIDE
    last = rand(1, 256, 20480)
    w[-1, -256:] = last
    codes, scales = fg.quantize_weight("fp8_block128", w)
    want, want_scales = fg.quantize_weight("fp8_block128", last)
    same(codes[-256:], want)
    same(scales[-2:], want_scales)
    del codes, scales
    codes, scales = fg.quantize_weight("fp8_block128", w, transpose=True)
    want, want_scales = fg.quantize_weight("fp8_block128", last, transpose=True)
    same(codes[-20480:, -256:], want)
    same(scales[-160:, -2:], want_scales)


def test_columns():
    rows, cols = 128 * 4100, 8320
    assert rows * cols > WIDE
    tail = rand(2, 128, cols)
    x = zeros(rows, cols, tail)
    want = fg.quantize_columns(tail)
    for order in (None, torch.arange(rows, dtype=torch.int32, device="cuda")):
        c = fg.quantize_columns(x, rows=order)
        same(c.data.view(cols // 128, -1, 1 << 14)[:, -2], want.data.view(cols // 128, -1, 1 << 14)[:, 0])
        same(c.sf.view(cols // 128, -1, 512)[:, -2], want.sf.view(cols // 128, -1, 512)[:, 0])


def test_checkpoint_and_its_gradient():
    rows, width = 128 * 2050, 8320
    assert rows * 2 * width > WIDE
    tail, dy_tail = rand(3, 128, 2 * width), rand(4, 128, width)
    x = zeros(rows, 2 * width, tail)
    for a, b in zip(fg.swiglu_checkpoint("mxfp8_b32", x), fg.swiglu_checkpoint("mxfp8_b32", tail)):
        same(a.view(rows, -1)[-128:], b.view(128, -1))
    _, _, saved, saved_scales = fg.swiglu_checkpoint("mxfp8_b32", x)
    _, _, few, few_scales = fg.swiglu_checkpoint("mxfp8_b32", tail)
    dy = zeros(rows, width, dy_tail)
    del x
    # with a weight for each row: every token has one choice, and lies where its slot says
    tokens = torch.arange(rows, dtype=torch.int32, device="cuda")
    r = fg.Routing(torch.full((rows, 1), 0.75, device="cuda"), torch.zeros(rows, 1, dtype=torch.int32, device="cuda"),
                   torch.tensor([0, rows], dtype=torch.int32, device="cuda"), tokens, tokens.view(-1, 1))
    s = fg.Routing(r.weights[:128], r.experts[:128], torch.tensor([0, 128], dtype=torch.int32, device="cuda"), tokens[:128],
                   r.slots[:128])
    got = fg.swiglu_backward("mxfp8_b32", dy, saved, saved_scales, routing=r, columns=True, plain=True)
    want = fg.swiglu_backward("mxfp8_b32", dy_tail, few, few_scales, routing=s, columns=True, plain=True)
    for a, b in ((got.codes, want.codes), (got.scales, want.scales), (got.dx, want.dx), (got.dweights, want.dweights)):
        same(a.view(rows, -1)[-128:], b.view(128, -1))
    for a, b in ((got.dx_columns, want.dx_columns), (got.act_columns, want.act_columns)):
        same(a.data.view(a.N // 128, -1, 1 << 14)[:, -2], b.data.view(a.N // 128, -1, 1 << 14)[:, 0])
        same(a.sf.view(a.N // 128, -1, 512)[:, -2], b.sf.view(a.N // 128, -1, 512)[:, 0])


@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, False)])
def test_wgrad(dtype, accumulate):
    experts, n, k = 82, 7168, 7424
    assert experts * n * k > WIDE
    x, y = rand(5, 150, n), rand(6, 150, k)
    offsets = ref.fixed_offsets([0] * (experts - 1) + [150])
    a, b = fg.quantize_columns(x, offsets), fg.quantize_columns(y, offsets)
    out = torch.zeros(experts, n, k, device="cuda") if accumulate else None
    out = fg.grouped_wgrad(a, b, offsets, out=out, accumulate=accumulate, dtype=dtype)
    one = ref.fixed_offsets([150])
    same(out[-1], fg.grouped_wgrad(fg.quantize_columns(x, one), fg.quantize_columns(y, one), one, dtype=dtype)[0])
    assert not out[:-1].any()


def test_wgrad_of_large_operands():
    """The images pass 2^32 bytes; the last expert's rows lie at their ends."""
    rows, n = 128 * 4100, 8320
    tail = rand(7, 128, n)
    offsets = ref.fixed_offsets([rows - 128, 128])
    a = fg.quantize_columns(zeros(rows, n, tail), offsets)
    assert a.data.numel() > WIDE
    b = fg.quantize_columns(zeros(rows, 128, tail[:, :128]), offsets)
    got = fg.grouped_wgrad(a, b, offsets)
    one = ref.fixed_offsets([128])
    same(got[1], fg.grouped_wgrad(fg.quantize_columns(tail), fg.quantize_columns(tail[:, :128].contiguous()), one)[0])
    assert not got[0].any()


def test_router():
    tokens, experts = 1 << 24, 264
    assert tokens * experts > WIDE
    tail = rand(8, 40, experts)
    logits = zeros(tokens, experts, tail)
    chosen = torch.zeros(tokens, 1, dtype=torch.int32, device="cuda")
    dw = torch.ones(tokens, 1, device="cuda")
    slopes = torch.randn(experts, device="cuda")
    r = fg.Routing(dw, chosen, None, None, None)
    s = fg.Routing(dw[:40], chosen[:40], None, None, None)
    got = fg.moe_route_backward(logits, r, dw, slopes, renormalize=False)
    same(got[-40:], fg.moe_route_backward(tail, s, dw[:40], slopes, renormalize=False))
    del got
    offsets = torch.arange(experts + 1, dtype=torch.int32, device="cuda")
    p = fg.moe_balance_loss(logits, offsets).probs.double()
    want = (torch.softmax(tail.double(), 1).sum(0) + (tokens - 40) / experts) / tokens
    # a warp adds up T / (152 * 32) + 1 tokens one by one, each rounded once; then 32 warps and 152 blocks
    steps = tokens / (152 * 32) + 32 + 152 + 8
    assert ((p - want).abs() <= steps * 2.0 ** -24 * want).all()


def test_grouped_block():
    rows, n, k = 128 * 4100, 8320, 128
    assert rows * n > WIDE
    pb = fg.preshuffle_b("fp8_block128", *fg.quantize_weight("fp8_block128", rand(9, n, k)))
    a, a_s = fg.quantize("fp8_block128", zeros(rows, k, rand(10, 300, k)))
    got = fg.grouped_gemm(a, pb, ref.fixed_offsets([rows]), a_s)
    want = fg.grouped_gemm(a[-300:].contiguous(), pb, ref.fixed_offsets([300]), a_s[-300:].contiguous())
    same(got[-300:], want)
    assert not got[:-300].any()
