"""Grouped products in fp8_block128 about where the form changes between 32-row and
128-row tiles, by rows, width and gathering: the bound of test_gpu_grouped.py, exact
sums, rows of no expert, and workspaces of the size that is asked for."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests.test_gpu_grouped import Experts, assert_close

pytestmark = pytest.mark.gpu

# 128-row tiles gathered too, and then some that take them only in place, or not at all (one weight tile, few rows)
WIDE = [
    ([65, 200, 0, 129, 128, 127, 1, 300], 2048, 1024),
    ([64, 65, 63, 256, 0, 0, 257, 90], 2176, 640),     # an odd count of weight tiles and of K steps
    ([600], 4096, 256),
    ([34] * 64, 640, 512),
]
NARROW = [([1000] * 4, 256, 1024), ([500] * 16, 128, 1024), ([100] * 33, 128, 640), ([70, 0, 300, 33], 128, 128)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k", WIDE + NARROW)
def test_against_64_bits(counts, n, k, gather):
    c = Experts("fp8_block128", counts, n, k, n + k, gather_from=77 if gather else None)
    y = c.run()
    assert_close(y, c.reference(), counts)
    size = fg.grouped_gemm_workspace_size("fp8_block128", c.r, len(counts), n, k, gather)
    buf = torch.full((size + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    again = torch.empty_like(y)
    c.run(Y=again, workspace=buf[:size])
    assert torch.equal(y, again) and (buf[size:] == 0xa5).all()


@pytest.mark.parametrize("counts,n,k", WIDE[:3])
def test_gathered_and_in_place_give_the_same_bits(counts, n, k):
    c = Experts("fp8_block128", counts, n, k, 3, gather_from=50)
    y = c.run()
    rows = c.rows.long()
    laid = fg.grouped_gemm(c.a[rows].contiguous(), c.pb, c.offsets, c.a_s[rows].contiguous())
    assert torch.equal(laid, y)


def test_rows_of_no_expert_stay():
    c = Experts("fp8_block128", [200] * 8, 2048, 512, 4, gather_from=60)
    cuts = [100, 300, 300, 250, 700, 900, 1300, 1290, 1500]      # begins late, ends early, decreases
    c.offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    y = torch.full((c.r, 2048), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(Y=y)
    assert (y[:100] == 3).all() and (y[1500:] == 3).all()
    c.offsets = torch.tensor([100, 300, 300, 300, 700, 900, 1300, 1300, 1500], dtype=torch.int32, device="cuda")
    want = c.reference()[100:1500]
    rms = want.pow(2).mean(1, keepdim=True).sqrt()
    assert ((y[100:1500].double() - want).abs() <= 2e-3 * rms + 2.0 ** -8 * want.abs()).all()


def test_a_call_that_ran_out_of_time_gathered():
    c = Experts("fp8_block128", [150, 200, 90, 300], 4096, 2048, 6, gather_from=80)
    want = c.run()
    torch.cuda.synchronize()
    fg.set_wait_timeout_ns(20_000_000)
    try:
        c.run(flags=fg.FG_FLAG_DEBUG_STALL)
        assert fg.get_error() == fg.FG_ERR_TIMEOUT
    finally:
        fg.set_wait_timeout_ns(4_000_000_000)
    assert torch.equal(c.run(), want) and fg.get_error() == fg.FG_OK


@pytest.mark.parametrize("counts,n,k", WIDE + NARROW)
def test_gathered_without_room_for_the_rows(counts, n, k):
    """The workspace of a call that gathers nothing is enough; one byte less is refused."""
    c = Experts("fp8_block128", counts, n, k, n + k, gather_from=77)
    size = fg.grouped_gemm_workspace_size("fp8_block128", c.r, len(counts), n, k, False)
    buf = torch.full((size + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    y = c.run(workspace=buf[:size])
    assert_close(y, c.reference(), counts)
    assert (buf[size:] == 0xa5).all()
    with pytest.raises(fg.FgError, match="workspace"):
        c.run(workspace=buf[:size - 1])
