"""The grouped product's form for many rows an expert: token tiles of up to 256
rows on pairs of SMs, in every mode that has it, and the 32-row form where the
rows lie on few of many experts.  Each test says which form runs.

Bounds are those of tests/test_gpu_grouped.py.
"""
import numpy as np
import pytest
import torch

import mx_gemm_gb300 as fg
from tests.test_gpu_grouped import MODES, Experts, assert_close

pytestmark = pytest.mark.gpu

PAIR_MODES = [m for m in MODES if m != "fp8_block128"]


def on_pairs(c, k):
    """Whether the call runs on pairs of SMs: only there do gathered rows take space."""
    size = [fg.grouped_gemm_workspace_size(c.mode, c.r, len(c.offsets) - 1, c.n, k, gather) for gather in (False, True)]
    return size[1] > size[0]


def heavy(experts, rows, of):
    """Few experts of many hold most of the rows."""
    rng = np.random.default_rng(experts)
    counts = rng.integers(0, 3, experts)
    counts[rng.choice(experts, of, replace=False)] += rows // of
    return counts.tolist()


# counts, weight rows of an expert, K
RAGGED = {
    # widths around 32, 64, 128, 160, 256 and their multiples; eleven weight tiles (the last pair's odd SM idles)
    "widths": ([128, 129, 160, 161, 192, 193, 255, 256, 257, 1, 31, 32, 33, 0, 511, 512, 513, 64, 65, 96, 97, 7], 1408, 1280),
    "prefill": ([255, 256, 257, 1, 0, 511, 513, 300], 1152, 768),
    "skewed": ([0, 0, 2000, 0, 0, 5, 1, 0, 700, 0], 640, 1792),
    "one_weight_tile": ([1000] * 8 + [3], 128, 256),          # one K step in mxfp4
    "long": ([300, 17, 0, 450, 1100, 2], 1280, 4096),
    "many_experts": (heavy(256, 3000, 7), 256, 2560),
}


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("mode", PAIR_MODES)
@pytest.mark.parametrize("name", list(RAGGED))
def test_ragged(mode, name, gather):
    counts, n, k = RAGGED[name]
    c = Experts(mode, counts, n, k, n + k, gather_from=777 if gather else None)
    assert on_pairs(c, k)
    assert_close(c.run(), c.reference(), (mode, name))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("mode", MODES)
def test_few_experts_of_many_in_the_32_row_form(mode, gather):
    """256 experts, 2048 rows at most: one expert's rows run as tens of tiles."""
    for of in (1, 5):
        c = Experts(mode, heavy(256, 1500, of), 256, 2560, of, gather_from=400 if gather else None)
        assert not on_pairs(c, 2560)
        assert_close(c.run(), c.reference(), (mode, of))


@pytest.mark.parametrize("mode", ["mxfp8_b32", "fp8_block128", "bf16"])
def test_units_shared_at_both_ends(mode):
    """The 32-row form's cut line: more units than blocks, K steps that do not divide, and units over three blocks."""
    for counts, n, k in (([3, 1, 0, 9, 2, 2, 7, 8] * 4, 1408, 7168 if mode != "bf16" else 3584), ([5, 0, 30], 128, 7168)):
        c = Experts(mode, counts, n, k, 5, gather_from=20)
        assert not on_pairs(c, k)
        assert_close(c.run(), c.reference(), (mode, n))


def case(mode, seed, gather_from=None):
    """Eight experts of 510 rows (tiles of 256 and 254), three weight tiles each, in more units than pairs."""
    c = Experts(mode, [510] * 8, 1408, 1024, seed, gather_from=gather_from)
    assert on_pairs(c, 1024)
    return c


@pytest.mark.parametrize("mode", PAIR_MODES)
def test_rows_no_expert_holds_are_left(mode):
    c = case(mode, 9)
    ref = c.reference()
    lo, hi = 5, c.r - 300
    c.offsets = c.offsets.clamp(lo, hi)
    y = torch.full((c.r, c.n), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(Y=y)
    assert (y[:lo] == 3).all() and (y[hi:] == 3).all()
    assert_close(y[lo:hi], ref[lo:hi], "held rows")


@pytest.mark.parametrize("mode", ["bf16", "mxfp8_b32", "mxfp4"])
def test_offsets_and_rows_out_of_range_stay_in_bounds(mode):
    c = case(mode, 10, gather_from=30)
    rows, offsets = c.rows.clone(), c.offsets.clone()
    c.rows[3], c.rows[7], c.rows[-1] = -5, 1 << 30, 30
    rows[3], rows[7], rows[-1] = 0, 29, 29
    c.offsets[0], c.offsets[8] = -100, 1 << 30
    y = c.run()
    c.rows, c.offsets = rows, offsets
    assert_close(y, c.reference(), "clamped")


@pytest.mark.parametrize("mode", PAIR_MODES)
def test_same_bits_each_time_and_beside_other_rows(mode):
    c = case(mode, 11)
    first = c.run()
    ws = torch.randint(0, 256, (fg.grouped_gemm_workspace_size(mode, c.r, 8, c.n, 1024) + 16,), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(c.run(workspace=ws), first)
    nan = c.a.clone()
    s = c.a_s
    if mode == "bf16":
        nan[1] = float("nan")
    elif mode == "mxfp4":                  # (its elements have no NaN)
        s = c.a_s.view(torch.uint8).clone()
        s[1] = 255
    else:
        nan.view(torch.uint8)[1] = 0x7f
    other = fg.grouped_gemm(nan, c.pb, c.offsets, s)
    keep = torch.arange(c.r, device="cuda") != 1
    assert torch.isnan(other[1]).all() and torch.equal(other[keep], first[keep])


@pytest.mark.parametrize("mode", ["mxfp8", "mxfp8_b32", "mxfp4", "mxfp4_fp8a"])
def test_scales_that_are_not_aligned(mode):
    c = case(mode, 13, gather_from=100)
    buf = torch.zeros(c.a_s.numel() + 1, dtype=torch.uint8, device="cuda")
    odd = buf[1:].view(c.a_s.shape)
    odd.copy_(c.a_s.view(torch.uint8))
    assert torch.equal(fg.grouped_gemm(c.a, c.pb, c.offsets, odd, rows=c.rows), c.run())


@pytest.mark.parametrize("mode", PAIR_MODES)
def test_graph_replay(mode):
    c = case(mode, 15, gather_from=600)
    want = c.run()
    y = torch.zeros_like(want)
    ws = torch.empty(fg.grouped_gemm_workspace_size(mode, c.r, 8, c.n, 1024, True) + 16, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(Y=y, workspace=ws)
    for _ in range(3):
        y.zero_()
        graph.replay()
        assert torch.equal(y, want)


def test_calls_one_after_the_other_on_two_streams():
    a, b = case("mxfp8_b32", 17, gather_from=16), case("bf16", 18)
    want = a.run(), b.run()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = [(a.run(stream=other), b.run()) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in got)


@pytest.mark.parametrize("mode", ["mxfp8_b32", "mxfp4", "mxfp4_fp8a", "bf16"])
def test_a_wait_that_runs_out_is_reported(mode):
    """With the MMA issuer held back both SMs' waits give up, the copies under way land, and the next call is sound."""
    c = case(mode, 16)
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
