"""Grouped products in fp8_block128 with many rows an expert (128-row tiles): the
bound of test_gpu_grouped.py, exact sums of whole numbers, and the same bits as the
32-row form's."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests.test_gpu_grouped import Experts, assert_close, values

pytestmark = pytest.mark.gpu

# many rows: over 32 an expert, and units (row tiles x pairs of weight tiles) for a third of the SMs
CASES = [
    ([65, 200, 0, 129, 128, 127, 1, 300], 1024, 1024),
    ([40] * 8 + [0] * 2 + [700], 1024, 128),           # one K step
    ([64, 65, 63, 256, 0, 0, 257, 90], 1152, 384),     # an odd count of weight tiles, steps that are no multiple of four
    ([100] * 33, 128, 640),                            # one weight tile
    ([1500], 1024, 2048),
    ([34] * 64, 256, 512),
]


def many(c, n, k):
    return c.r > 32 * (len(c.offsets) - 1) and (c.r // 128 + min(len(c.offsets) - 1, c.r)) * ((n // 128 + 1) // 2) >= 48


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k", CASES)
def test_against_64_bits(counts, n, k, gather):
    c = Experts("fp8_block128", counts, n, k, n + k, gather_from=77 if gather else None)
    assert many(c, n, k)
    assert_close(c.run(), c.reference(), counts)


@pytest.mark.parametrize("gather", [False, True])
def test_exact(gather):
    """Whole numbers and scales that are powers of two: every sum is exact."""
    g = torch.Generator(device="cuda").manual_seed(1)
    counts, n, k = [150, 0, 33, 128, 400, 1, 60, 90], 640, 768
    c = Experts("fp8_block128", counts, n, k, 2, gather_from=50 if gather else None)
    whole = torch.randint(-3, 4, c.a.shape, generator=g, device="cuda").float()
    c.a, c.a_s = whole.to(torch.float8_e4m3fn), torch.exp2(torch.randint(-1, 2, c.a_s.shape, generator=g, device="cuda").float())
    b = torch.randint(-3, 4, c.b.shape, generator=g, device="cuda").float()
    c.b, c.b_s = b.to(torch.float8_e4m3fn), torch.exp2(torch.randint(-1, 2, c.b_s.shape, generator=g, device="cuda").float())
    c.pb = fg.preshuffle_b("fp8_block128", c.b, c.b_s)
    y = torch.full((c.r, n), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(c.run(Y=y), c.reference().to(torch.bfloat16))


def test_the_bits_of_the_32_row_form():
    """Up to twelve K steps the line of the 32-row form is not cut: a row alone has the bits it has among many."""
    c = Experts("fp8_block128", [150, 200, 90, 300], 1024, 1024, 3)
    y, cuts = c.run(), c.offsets.tolist()
    for at in (0, 149, 150, 349, 350, 439, 440, 739):
        e = max(i for i in range(4) if cuts[i] <= at)
        one = torch.tensor([0] * (e + 1) + [1] * (4 - e), dtype=torch.int32, device="cuda")
        few = fg.grouped_gemm(c.a[at:at + 1].contiguous(), c.pb, one, c.a_s[at:at + 1].contiguous())
        assert torch.equal(few[0], y[at]), at


@pytest.mark.parametrize("gather", [False, True])
def test_rows_of_no_expert_stay_and_nothing_is_written_past_the_workspace(gather):
    c = Experts("fp8_block128", [200] * 8, 1024, 512, 4, gather_from=60 if gather else None)
    want = c.run()
    cuts = [100, 300, 300, 250, 700, 900, 1300, 1290, 1500]      # begins late, ends early, decreases
    c.offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    size = fg.grouped_gemm_workspace_size("fp8_block128", c.r, 8, 1024, 512, gather)
    buf = torch.full((size + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    y = torch.full((c.r, 1024), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(Y=y, workspace=buf[:size])
    assert (buf[size:] == 0xa5).all() and (y[:100] == 3).all() and (y[1500:] == 3).all()
    clean = [100, 300, 300, 300, 700, 900, 1300, 1300, 1500]
    c.offsets = torch.tensor(clean, dtype=torch.int32, device="cuda")
    ref = c.reference()
    rms = ref[100:1500].pow(2).mean(1, keepdim=True).sqrt()
    assert ((y[100:1500].double() - ref[100:1500]).abs() <= 2e-3 * rms + 2.0 ** -8 * ref[100:1500].abs()).all()
    assert want.shape == y.shape


def test_values_that_are_not_numbers_stay_in_their_rows():
    c = Experts("fp8_block128", [150, 200, 90, 300], 1024, 512, 5)
    want = c.run()
    c.a_s = c.a_s.clone()
    c.a_s[160, 1] = float("nan")
    y = c.run()
    bad = torch.zeros(c.r, dtype=torch.bool, device="cuda")
    bad[160] = True
    assert torch.equal(torch.isnan(y), bad[:, None].expand_as(y))
    assert torch.equal(y[~bad], want[~bad])


def test_a_call_that_ran_out_of_time_and_its_replay():
    c = Experts("fp8_block128", [150, 200, 90, 300], 1024, 2048, 6)
    want = c.run()
    torch.cuda.synchronize()
    fg.set_wait_timeout_ns(20_000_000)
    try:
        c.run(flags=fg.FG_FLAG_DEBUG_STALL)
        assert fg.get_error() == fg.FG_ERR_TIMEOUT
    finally:
        fg.set_wait_timeout_ns(4_000_000_000)
    assert torch.equal(c.run(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = c.run()
    for _ in range(3):
        y.zero_()
        graph.replay()
        assert torch.equal(y, want)
    assert fg.get_error() == fg.FG_OK


def test_scales_at_any_address_and_operands_as_bytes():
    c = Experts("fp8_block128", [150, 200, 90, 300], 1024, 1024, 7)
    want = c.run()
    buf = torch.empty(c.a_s.numel() + 1, device="cuda")
    buf[1:] = c.a_s.flatten()
    c.a_s = buf[1:].view(c.a_s.shape)                            # 4 bytes past a 16-byte boundary
    c.a = c.a.view(torch.uint8)
    assert torch.equal(c.run(), want)
    assert values(c.a, c.a_s, "fp8_block128").isfinite().all()
