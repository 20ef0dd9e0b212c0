"""Products grouped by expert against the 64-bit product of the operands that
the codes stand for.

Bound of an output: fp32 accumulation over K terms of 8 / 4-bit products (and
the tensor core's own alignment of addends) within the parity bound that the
library's GEMM is held to, 2e-3 of the root mean square here, and half a bf16
step of the value, 2^-8, for the rounding.
"""
import numpy as np
import pytest
import torch

import mx_gemm_gb300 as fg
import oracle

pytestmark = pytest.mark.gpu

MODES = ("bf16", "fp8_tensor", "fp8_block128", "mxfp8", "mxfp8_b32", "mxfp4", "mxfp4_fp8a")


def values(codes, scales, mode):
    """fp64 values [rows][K] on the GPU of codes and scales."""
    if mode == "bf16":
        return codes.double()
    c = codes.view(torch.uint8).long()
    if mode == "mxfp4":
        table = torch.from_numpy(oracle.table_e2m1()).cuda()
        v = torch.stack((table[c & 15], table[c >> 4]), dim=2).flatten(1)
    else:
        v = torch.from_numpy(oracle.table_e4m3()).cuda()[c]
    if mode == "fp8_tensor":
        return v * scales.double()
    if mode == "fp8_block128":  # [rows][K/128], or a weight's [rows/128][K/128]
        s = scales.double().repeat_interleave(v.shape[0] // scales.shape[0], 0)
        return (v.unflatten(1, (s.shape[1], -1)) * s[:, :, None]).flatten(1)
    s = torch.from_numpy(oracle.table_e8m0()).cuda()[scales.view(torch.uint8).long()]
    return (v.unflatten(1, (s.shape[1], -1)) * s[:, :, None]).flatten(1)


def operand(x, mode, weight=False):
    """(codes, scales, mode the values are read by) of fp32 x."""
    if mode == "bf16":
        return x.to(torch.bfloat16), None, mode
    if mode == "fp8_tensor":
        s = (x.abs().max() / 448).reshape(1)
        return (x / s).to(torch.float8_e4m3fn), s, mode
    if mode == "fp8_block128" and weight:
        b = x.view(x.shape[0] // 128, 128, -1, 128)
        s = b.abs().amax((1, 3)) / 448
        return (b / s[:, None, :, None]).view(x.shape).to(torch.float8_e4m3fn), s, mode
    m = "mxfp4" if weight and mode == "mxfp4_fp8a" else mode
    c, s = fg.quantize(m, x)
    return c, s, m


class Experts:
    """E stacked weights [N][K], T rows of A, offsets from counts."""

    def __init__(self, mode, counts, n, k, seed, gather_from=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.mode, self.n = mode, n
        self.r, e = sum(counts), len(counts)
        self.t = self.r if gather_from is None else gather_from
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        rough = torch.exp2(torch.randint(-3, 4, (max(self.t, 1), k // 64), generator=g, device="cuda").float())
        a = torch.randn(max(self.t, 1), k, generator=g, device="cuda") * rough.repeat_interleave(64, 1)
        self.a, self.a_s, self.am = operand(a, mode)
        b = torch.randn(e * n, k, generator=g, device="cuda") * torch.exp2(
            torch.randint(-2, 3, (e * n, 1), generator=g, device="cuda").float())
        self.b, self.b_s, self.bm = operand(b, mode, weight=True)
        self.pb = fg.preshuffle_b(mode, self.b, self.b_s, K=k)
        self.rows = None
        if gather_from is not None:
            self.rows = torch.randint(0, self.t, (self.r,), generator=g, device="cuda", dtype=torch.int32)

    def run(self, **kw):
        return fg.grouped_gemm(self.a, self.pb, self.offsets, self.a_s, rows=self.rows, **kw)

    def reference(self):
        a, b = values(self.a, self.a_s, self.am), values(self.b, self.b_s, self.bm)
        if self.rows is not None:
            a = a[self.rows.long()]
        out = torch.zeros(self.r, self.n, dtype=torch.float64, device="cuda")
        cuts = self.offsets.tolist()
        for e in range(len(cuts) - 1):
            out[cuts[e]:cuts[e + 1]] = a[cuts[e]:cuts[e + 1]] @ b[e * self.n:(e + 1) * self.n].T
        return out


def assert_close(y, ref, what):
    rms = ref.pow(2).mean(1, keepdim=True).sqrt()  # a row's own: rows differ in size
    bad = (y.double() - ref).abs() > 2e-3 * rms + 2.0 ** -8 * ref.abs()
    assert not bad.any(), (what, int(bad.sum()), (y.double() - ref).abs().max().item())
    assert fg.get_error() == fg.FG_OK


RAGGED = {
    "one_row": [0, 0, 1, 0],
    "decode": [1, 0, 3, 16, 17, 0, 0, 2, 31, 32, 33, 5],
    "one_expert": [7],
    "few": [100, 0, 129],
    "prefill": [255, 256, 257, 1, 0, 511, 513, 300],
    "skewed": [0, 1500, 0, 0, 3, 0, 1, 0],
    "all_of_one": [0, 0, 0, 65],
}


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shape", [(128, 256), (384, 768), (256, 2048), (640, 1280)])
@pytest.mark.parametrize("counts", list(RAGGED))
def test_ragged(mode, counts, shape, gather):
    n, k = shape
    c = Experts(mode, RAGGED[counts], n, k, n + k + len(counts), gather_from=77 if gather else None)
    assert_close(c.run(), c.reference(), (mode, counts, shape))


@pytest.mark.parametrize("mode", MODES)
def test_long_rows_and_many_units(mode):
    """Every block shares units at both ends: more units than blocks, K steps that do not divide."""
    c = Experts(mode, [3, 1, 0, 9, 40, 2, 16, 8] * 4, 2048, 7168 if mode != "bf16" else 3584, 5, gather_from=20)
    assert_close(c.run(), c.reference(), mode)


@pytest.mark.parametrize("mode", ["mxfp8_b32", "mxfp4"])
def test_most_experts(mode):
    counts = np.random.default_rng(1).integers(0, 3, 1024).tolist()
    c = Experts(mode, counts, 128, 256, 6)
    assert_close(c.run(), c.reference(), mode)
    many = np.random.default_rng(2).integers(0, 60, 1024).tolist()
    c = Experts(mode, many, 128, 256, 7)
    assert_close(c.run(), c.reference(), mode)


@pytest.mark.parametrize("total", [40, 2000])
def test_rows_no_expert_holds_are_left(total):
    c = Experts("mxfp8_b32", [total // 4] * 4, 256, 512, 9)
    ref = c.reference()
    lo, hi = 5, total - 7
    c.offsets = c.offsets.clamp(lo, hi)
    y = torch.full((total, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(Y=y)
    assert (y[:lo] == 3).all() and (y[hi:] == 3).all()
    assert_close(y[lo:hi], ref[lo:hi], "held rows")


@pytest.mark.parametrize("total", [40, 2000])
def test_offsets_and_rows_out_of_range_stay_in_bounds(total):
    """Offsets are clamped into 0..R and rows into 0..T-1: the call computes what the clamped ones say."""
    c = Experts("mxfp8_b32", [total // 4] * 4, 256, 512, 10, gather_from=30)
    rows = c.rows.clone()
    c.rows[3], c.rows[7], c.rows[total - 1] = -5, 1 << 30, 30
    rows[3], rows[7], rows[total - 1] = 0, 29, 29
    offsets = c.offsets.clone()
    c.offsets[0], c.offsets[4] = -100, 1 << 30
    y = c.run()
    c.rows, c.offsets = rows, offsets
    assert_close(y, c.reference(), "clamped")


@pytest.mark.parametrize("mode,total", [("mxfp8_b32", 24), ("mxfp8_b32", 900), ("fp8_block128", 40)])
def test_same_bits_each_time_and_beside_other_rows(mode, total):
    """The same call gives the same bits, and a row's result does not depend on its neighbours'."""
    c = Experts(mode, [total // 8] * 8, 512, 4096, 11)
    first = c.run()
    ws = torch.randint(0, 256, (fg.grouped_gemm_workspace_size(mode, total, 8, 512, 4096) + 16,),
                       dtype=torch.uint8, device="cuda")[:]  # any contents
    for _ in range(5):
        assert torch.equal(c.run(workspace=ws), first)
    nan = c.a.view(torch.uint8).clone()
    nan[1] = 0x7f                      # a row of NaN codes
    other = fg.grouped_gemm(nan, c.pb, c.offsets, c.a_s)
    assert torch.isnan(other[1]).all()
    keep = torch.arange(c.r, device="cuda") != 1
    assert torch.equal(other[keep], first[keep])


def test_not_a_number_scales_reach_only_their_row():
    c = Experts("mxfp4", [3, 4], 128, 512, 12)
    first = c.run()
    s = c.a_s.view(torch.uint8).clone()
    s[2, 5] = 255
    y = fg.grouped_gemm(c.a, c.pb, c.offsets, s)
    assert torch.isnan(y[2]).all() and torch.equal(y[[0, 1, 3, 4, 5, 6]], first[[0, 1, 3, 4, 5, 6]])


def test_scales_that_are_not_word_aligned():
    c = Experts("mxfp8_b32", [9, 20, 1], 256, 1024, 13)
    buf = torch.zeros(c.a_s.numel() + 1, dtype=torch.uint8, device="cuda")
    odd = buf[1:].view(c.a_s.shape)
    odd.copy_(c.a_s.view(torch.uint8))
    assert torch.equal(fg.grouped_gemm(c.a, c.pb, c.offsets, odd), c.run())


def test_no_rows():
    c = Experts("mxfp8_b32", [4, 4], 128, 256, 14)
    empty = c.a[:0]
    y = fg.grouped_gemm(empty, c.pb, torch.zeros(3, dtype=torch.int32, device="cuda"), c.a_s[:0])
    assert y.shape == (0, 128)
    y = torch.full((8, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    fg.grouped_gemm(c.a, c.pb, torch.zeros(3, dtype=torch.int32, device="cuda"), c.a_s, Y=y)
    assert (y == 2).all()


@pytest.mark.parametrize("total", [24, 900])
def test_graph_replay(total):
    c = Experts("mxfp8_b32", [total // 8] * 8, 512, 4096, 15)
    want = c.run()
    y = torch.zeros_like(want)
    ws = torch.empty(fg.grouped_gemm_workspace_size("mxfp8_b32", total, 8, 512, 4096) + 16, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(Y=y, workspace=ws)
    for _ in range(4):
        y.zero_()
        graph.replay()
        assert torch.equal(y, want)


@pytest.mark.parametrize("mode,total", [("mxfp8_b32", 24), ("mxfp8_b32", 900), ("fp8_block128", 24)])
def test_a_wait_that_runs_out_is_reported(mode, total):
    """With the MMA issuer held back every wait gives up and the call ends in FG_ERR_TIMEOUT; the next call is sound."""
    c = Experts(mode, [total // 8] * 8, 512, 4096, 16)
    want = c.run()
    torch.cuda.synchronize()
    fg.set_wait_timeout_ns(20_000_000)
    try:
        c.run(flags=fg.FG_FLAG_DEBUG_STALL)
        assert fg.get_error() == fg.FG_ERR_TIMEOUT
    finally:
        fg.set_wait_timeout_ns(4_000_000_000)
    assert torch.equal(c.run(), want)
    assert fg.get_error() == fg.FG_OK


@pytest.mark.parametrize("gather", [True, False])
def test_outputs_past_32_bits_of_elements(gather):
    """Y beyond element 2^31: the first and last rows against the reference."""
    total, experts, n, k = 540_000, 8, 4096, 256
    c = Experts("mxfp8_b32", [total // experts] * experts, n, k, 21, gather_from=500 if gather else None)
    y = c.run()
    b = values(c.b, c.b_s, c.bm)
    for rows, e in ((slice(0, 40), 0), (slice(total - 40, total), experts - 1)):
        at = c.rows[rows].long() if gather else torch.arange(total, device="cuda")[rows]
        mine = values(c.a.view(torch.uint8)[at].view(c.a.dtype), c.a_s.view(torch.uint8)[at], c.am)
        assert_close(y[rows], mine @ b[e * n:(e + 1) * n].T, rows)


@pytest.mark.parametrize("total", [24, 1200])
def test_another_stream(total):
    c = Experts("mxfp8_b32", [total // 8] * 8, 512, 4096, 17, gather_from=16)
    want = c.run()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = [c.run(stream=other) for _ in range(3)]
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]  # would reuse a freed workspace
    torch.cuda.current_stream().wait_stream(other)
    assert all(torch.equal(y, want) for y in got) and len(junk) == 8


@pytest.mark.parametrize("total", [24, 1200])
def test_units_and_tiles_do_not_change_a_row(total):
    """A row's bits are the same whatever expert counts surround it, in either form."""
    c = Experts("mxfp8_b32", [total // 8] * 8, 256, 1024, 18)
    first = c.run()
    # the same rows of expert 3, alone
    lo, hi = 3 * (total // 8), 4 * (total // 8)
    one = torch.zeros(9, dtype=torch.int32, device="cuda")
    one[4:] = hi - lo
    y = fg.grouped_gemm(c.a[lo:hi].contiguous(), c.pb, one, c.a_s[lo:hi].contiguous())
    diff = (y.double() - first[lo:hi].double()).abs()
    assert (diff <= 2.0 ** -7 * first[lo:hi].double().abs() + 1e-3 * first.double().pow(2).mean().sqrt()).all()


@pytest.mark.parametrize("edit,text", [
    (dict(offsets="long"), "offsets"), (dict(offsets="few"), "divisor"), (dict(a="float"), "A has dtype"), (dict(a="wide"), "A must be"),
    (dict(rows="long"), "rows"), (dict(scales="short"), "a_scales"), (dict(scales="float"), "a_scales"), (dict(Y="shape"), "Y has"),
    (dict(Y="float"), "Y has"), (dict(workspace="host"), "workspace"),
])
def test_binding_refusals(edit, text):
    c = Experts("mxfp8_b32", [4, 4, 4], 128, 256, 19, gather_from=12)
    kw = dict(A=c.a, pb=c.pb, offsets=c.offsets, a_scales=c.a_s, rows=c.rows)
    what, how = next(iter(edit.items()))
    kw.update({("offsets", "long"): dict(offsets=c.offsets.long()), ("offsets", "few"): dict(offsets=torch.zeros(6, dtype=torch.int32, device="cuda")),
               ("a", "float"): dict(A=c.a.float()), ("a", "wide"): dict(A=c.a[:, :128].contiguous()), ("rows", "long"): dict(rows=c.rows.long()),
               ("scales", "short"): dict(a_scales=c.a_s[:5].contiguous()), ("scales", "float"): dict(a_scales=c.a_s.float()),
               ("Y", "shape"): dict(Y=torch.empty(12, 256, dtype=torch.bfloat16, device="cuda")),
               ("Y", "float"): dict(Y=torch.empty(12, 128, device="cuda")), ("workspace", "host"): dict(workspace=torch.empty(8))}[(what, how)])
    with pytest.raises(ValueError, match=text):
        fg.grouped_gemm(**kw)


def test_library_refusals_come_as_errors():
    c = Experts("mxfp8_b32", [4, 4, 4], 128, 256, 20)
    with pytest.raises(fg.FgError) as e:
        c.run(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == fg.FG_ERR_WORKSPACE
    with pytest.raises(fg.FgError) as e:
        c.run(flags=1)
    assert e.value.status == fg.FG_ERR_INVALID_ARG
