"""Quantisation of activations and RMS norm with quantised output.

Without the gated activation the operator only rounds, so codes and scales
are compared for equality with the 64-bit recipe of `inputs`.  Where 32-bit
arithmetic comes first (the gated activation, the norm), each value that the
codes stand for is held to the 64-bit value within half a step of its format,
plus REL of the value for the arithmetic: at most 20 operations and two fast
functions of 2 ulp each, under 2^-18.
"""
import numpy as np
import pytest
import torch

import inputs
import mx_gemm_gb300 as fg
import oracle

pytestmark = pytest.mark.gpu

MX = ("mxfp8_b32", "mxfp8", "mxfp4", "mxfp4_fp8a")
REL = 2.0 ** -18


def block(mode):
    return 128 if mode in ("mxfp8", "fp8_block128") else 32


def fmt(mode):
    return "e2m1" if mode == "mxfp4" else "e4m3"


def code_bytes(codes):
    return codes.view(torch.uint8).cpu().numpy()


def decoded(codes, mode):
    """fp64 values of the codes, without their scales."""
    c = code_bytes(codes)
    if mode == "mxfp4":
        out = np.empty((c.shape[0], 2 * c.shape[1]))
        out[:, 0::2], out[:, 1::2] = oracle.table_e2m1()[c & 15], oracle.table_e2m1()[c >> 4]
        return out
    return oracle.table_e4m3()[c]


def reference(x, mode):
    """(values of the codes, scales) of fp64 x by the recipe: E8M0 codes, or fp32 for fp8_block128."""
    b = x.reshape(x.shape[0], -1, block(mode))
    amax = np.abs(b).max(axis=2)
    bad = ~np.isfinite(amax)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.where(bad, 0.0, amax)
    if mode == "fp8_block128":
        s = np.where(amax == 0, np.float32(1), amax.astype(np.float32) / np.float32(448)).astype(np.float32)
        q = (b.astype(np.float32) / s[:, :, None]).reshape(x.shape)
        return oracle.table_e4m3()[inputs.to_e4m3_codes(q)], np.where(bad, np.float32(np.nan), s)
    top = inputs.E2M1_MAX if mode == "mxfp4" else inputs.E4M3_MAX
    c = inputs.e8m0_for(amax, top)
    q = (b / np.ldexp(1.0, c.astype(np.int64) - 127)[:, :, None]).reshape(x.shape)
    v = oracle.table_e2m1()[inputs.to_e2m1_codes(q)] if mode == "mxfp4" else oracle.table_e4m3()[inputs.to_e4m3_codes(q)]
    return v, np.where(bad, 255, c).astype(np.uint8)


def rows_of(m, k, dtype, seed):
    """Values over many binades with the blocks a quantiser can go wrong at."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.exp2(torch.randint(-20, 20, (m, k // 32), generator=g).float()).repeat_interleave(32, 1)
    x = x.to(dtype)
    if m >= 8 and k >= 256:
        x[0, :32] = 0                      # a zero block beside others
        x[1, :] = 0                        # a zero row
        x[2, 5] = float("inf")
        x[3, 70] = float("nan")
        x[4, 3] = -float("inf")
        x[5, :128] = torch.finfo(dtype).tiny / 4  # subnormal
        x[5, 128:256] = 1e-38
        x[6, :128] = torch.finfo(dtype).max
        x[6, 128:160] = 448.0              # amax on the format's end: scale 1
        x[6, 160:192] = 6.0
        x[7, :32] = -0.0
        x[7, 32:64] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4).to(dtype)  # e2m1 ties
    return x


@pytest.mark.parametrize("mode", MX + ("fp8_block128",))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 128), (9, 256), (33, 7168), (130, 2944), (1000, 384)])
def test_codes_and_scales_are_exact(mode, dtype, m, k):
    x = rows_of(m, k, dtype, m + k)
    codes, scales = fg.quantize(mode, x.cuda())
    v, s = reference(x.double().numpy(), mode)
    if mode == "fp8_block128":
        assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    else:
        assert np.array_equal(code_bytes(scales), s)
    assert np.array_equal(decoded(codes, mode), v)


@pytest.mark.parametrize("mode", MX)
def test_narrowest_rows_and_row_distance(mode):
    """One block per row; rows that lie apart in a wider tensor, and rows of one row."""
    k = block(mode)
    wide = rows_of(37, 4 * k, torch.bfloat16, 3).cuda()
    for x in (wide[:, k:2 * k], wide[5:6, :k], wide[::2, :k]):
        codes, scales = fg.quantize(mode, x)
        v, s = reference(x.double().cpu().numpy(), mode)
        assert np.array_equal(code_bytes(scales), s) and np.array_equal(decoded(codes, mode), v)


def assert_stands_for(codes, scales, want, mode, what):
    """Scales are the recipe's for `want` or for a value REL away; values within half a step."""
    c = code_bytes(scales).astype(np.int64)
    amax = np.abs(want.reshape(want.shape[0], -1, block(mode))).max(axis=2)
    top = inputs.E2M1_MAX if mode == "mxfp4" else inputs.E4M3_MAX
    lo, hi = (inputs.e8m0_for(amax * f, top).astype(np.int64) for f in (1 - REL, 1 + REL))
    assert ((c >= lo) & (c <= hi)).all(), what
    s = np.repeat(np.ldexp(1.0, c - 127), block(mode), axis=1)
    got = decoded(codes, mode) * s
    man, low = (1, 0) if mode == "mxfp4" else (3, -6)   # fraction bits, exponent of the least normal
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(want) / s, 1e-300))), low)
    half = np.ldexp(0.5, (e - man).astype(np.int64)) * s
    assert (np.abs(got - want) <= half * (1 + 2.0 ** -10) + REL * np.abs(want) + 1e-37).all(), what


@pytest.mark.parametrize("mode", MX)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 128), (17, 2048), (300, 1408)])
def test_gated_activation(mode, dtype, m, k):
    g = torch.Generator().manual_seed(m + k)
    x = (3 * torch.randn(m, 2 * k, generator=g)).to(dtype)
    x[0, :4] = torch.tensor([-90.0, -30.0, 80.0, 0.0]).to(dtype)
    codes, scales = fg.quantize(mode, x.cuda(), act="swiglu")
    d = x.double().numpy()
    want = d[:, :k] / (1 + np.exp(-d[:, :k])) * d[:, k:]
    assert_stands_for(codes, scales, want, mode, (mode, m, k))


def test_gated_activation_keeps_what_is_not_finite():
    x = torch.ones(3, 512, dtype=torch.bfloat16, device="cuda")
    x[0, 3] = float("nan")
    x[1, 256 + 40] = float("inf")
    x[2, 7] = -float("inf")   # silu(-inf) = -inf / inf
    _, scales = fg.quantize("mxfp8_b32", x, act="swiglu")
    c = code_bytes(scales)
    assert (c == 255).tolist() == [[b == 0 for b in range(8)], [b == 1 for b in range(8)], [b == 0 for b in range(8)]]


@pytest.mark.parametrize("mode", MX)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k,residual", [(1, 7168, True), (5, 128, False), (200, 7168, True), (160, 2944, False),
                                          (3, 16384, True), (2, 32768, True), (400, 640, True)])
def test_rmsnorm(mode, dtype, m, k, residual):
    g = torch.Generator().manual_seed(k + m)
    x = torch.randn(m, k, generator=g).to(dtype)
    r = (5 * torch.randn(m, k, generator=g)).to(dtype) if residual else None
    w = (1 + 0.3 * torch.randn(k, generator=g)).to(dtype)
    codes, scales, h, y = fg.rmsnorm_quantize(mode, x.cuda(), w.cuda(), residual=None if r is None else r.cuda(),
                                              eps=1e-5, normed=True)
    h32 = x.float() + r.float() if residual else x.float()
    assert (h is None) == (r is None)
    if residual:
        assert torch.equal(h.cpu(), h32.to(dtype))
    h64 = x.double() + r.double() if residual else x.double()
    # a sum of k squares in chains of 32 and halving reductions: well under REL
    want = (h64 / torch.sqrt(h64.pow(2).mean(1, keepdim=True) + 1e-5) * w.double()).numpy()
    ulp = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    # h itself is rounded to 32 bits: |x| + |r| may exceed |h|
    slack = REL * np.abs(want) + 2.0 ** -22 * np.abs(want).max(axis=1, keepdims=True)
    assert (np.abs(y.double().cpu().numpy() - want) <= ulp * np.abs(want) + slack).all()
    assert_stands_for(codes, scales, want, mode, (mode, m, k))


def test_rmsnorm_without_codes_and_with_row_distance():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(50, 3 * 1000, generator=g).to(torch.bfloat16).cuda()
    w = torch.rand(1000, generator=g).to(torch.bfloat16).cuda()
    codes, scales, h, y = fg.rmsnorm_quantize("bf16", x[:, 1000:2000], w, residual=x[:, :1000])
    assert codes is None and scales is None
    hh = x[:, 1000:2000].float() + x[:, :1000].float()
    assert torch.equal(h, hh.to(torch.bfloat16))
    h64 = hh.double()
    want = h64 / torch.sqrt(h64.pow(2).mean(1, keepdim=True) + 1e-6) * w.double()
    assert ((y.double() - want).abs() <= (2.0 ** -8 + REL) * want.abs()).all()


def test_rmsnorm_zero_rows_and_not_finite_rows():
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    x[2, 9] = float("nan")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    codes, scales, _, y = fg.rmsnorm_quantize("mxfp8_b32", x, w, normed=True)
    c = code_bytes(scales)
    assert (c[0] == 127).all() and (code_bytes(codes)[0] == 0).all() and (y[0] == 0).all()
    assert (c[1] == 119).all() and (c[2] == 255).all() and torch.isnan(y[2]).all()


def test_fp8_block128_norm():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(20, 1024, generator=g).cuda()
    w = torch.ones(1024, device="cuda")
    codes, scales, _, y = fg.rmsnorm_quantize("fp8_block128", x, w, normed=True)
    v, s = reference(y.double().cpu().numpy(), "fp8_block128")  # y is the unrounded 32-bit result
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(decoded(codes, "fp8_block128"), v)


def test_quantised_operand_feeds_the_product():
    """quantize() gives fg.gemm its operands: against the product of the decoded values in 64 bits."""
    g = torch.Generator().manual_seed(4)
    a, b = torch.randn(5, 512, generator=g), torch.randn(256, 512, generator=g)
    for mode in MX:
        ca, sa = fg.quantize(mode, a.cuda())
        wmode = "mxfp4" if mode == "mxfp4_fp8a" else mode
        cb, sb = fg.quantize(wmode, b.cuda())
        y = fg.gemm(ca, fg.preshuffle_b(mode, cb, sb), sa).double().cpu().numpy()
        da, db = (decoded(c, m) * np.repeat(np.ldexp(1.0, code_bytes(s).astype(np.int64) - 127), block(m), axis=1)
                  for c, s, m in ((ca, sa, mode), (cb, sb, wmode)))
        want = da @ db.T
        assert np.abs(y - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-3, mode


def test_empty_and_other_stream():
    c, s = fg.quantize("mxfp8_b32", torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))
    assert c.shape == (0, 256) and s.shape == (0, 8)
    x = torch.randn(4096, 2048, device="cuda").to(torch.bfloat16)
    want = [code_bytes(t) for t in fg.quantize("mxfp8_b32", x)]
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = fg.quantize("mxfp8_b32", x, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert all(np.array_equal(code_bytes(a), b) for a, b in zip(got, want))


def test_rows_past_32_bits_of_elements():
    m, k = 270_000, 8192
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    edge = rows_of(16, k, torch.bfloat16, 5)
    x[:8], x[-8:] = edge[:8].cuda(), edge[8:].cuda()
    codes, scales = fg.quantize("mxfp8_b32", x)
    v, s = reference(edge.double().numpy(), "mxfp8_b32")
    take = torch.cat([torch.arange(8), torch.arange(m - 8, m)]).cuda()
    got = codes.view(torch.uint8)[take].view(torch.float8_e4m3fn)
    assert np.array_equal(decoded(got, "mxfp8_b32"), v)
    assert np.array_equal(scales.view(torch.uint8)[take].cpu().numpy(), s)
    del codes, scales
    w = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    x[-1] = 2.0
    _, _, _, y = fg.rmsnorm_quantize("bf16", x, w)
    assert ((y[-1].float() - 1).abs() < 2.0 ** -7).all() and (y[m // 2] == 0).all()


@pytest.mark.parametrize("call,text", [
    (lambda x: fg.quantize("mxfp8_b32", x.t()), "contiguous rows"),
    (lambda x: fg.quantize("mxfp8_b32", x.half()), "dtype"),
    (lambda x: fg.quantize("mxfp8_b32", x[0]), "2-D"),
    (lambda x: fg.quantize("mxfp8_b32", x[:, :255], act="swiglu"), "halves"),
    (lambda x: fg.quantize("mxfp8_b32", x[:1].expand(4, 256)), "overlapping"),
    (lambda x: fg.rmsnorm_quantize("mxfp8_b32", x, x[0, :128]), "weight"),
    (lambda x: fg.rmsnorm_quantize("mxfp8_b32", x, x[0].float()), "weight"),
    (lambda x: fg.rmsnorm_quantize("mxfp8_b32", x, x[0], residual=x[:2]), "residual"),
    (lambda x: fg.rmsnorm_quantize("mxfp8_b32", x, x[0], residual=x.float()), "residual"),
    (lambda x: fg.rmsnorm_quantize("mxfp8_b32", x, x[0], eps="a"), "eps"),
])
def test_binding_refusals(call, text):
    with pytest.raises(ValueError, match=text):
        call(torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"))


def test_library_refusals_come_as_errors():
    x = torch.zeros(4, 264, dtype=torch.bfloat16, device="cuda")
    for call, status in ((lambda: fg.quantize("mxfp8_b32", x), fg.FG_ERR_SHAPE),              # not whole blocks
                         (lambda: fg.quantize("fp8_tensor", x[:, :256]), fg.FG_ERR_INVALID_ARG),
                         (lambda: fg.quantize("mxfp8_b32", x[:, 1:257]), fg.FG_ERR_ALIGN)):    # rows 2 bytes off
        with pytest.raises(fg.FgError) as e:
            call()
        assert e.value.status == status
