"""What the grouped product's device data can do to its workspace: the offsets
are not seen by the host, so no values of theirs may move a store outside the
buffers or leave the workspace in a state that a later call trips over."""
import numpy as np
import pytest
import torch

import mx_gemm_gb300 as fg
from tests.test_gpu_grouped import Experts, assert_close

pytestmark = pytest.mark.gpu

GUARD = 1 << 20


def guarded(c, n, k, gather):
    """(the call's workspace, the guard bytes behind it)"""
    size = fg.grouped_gemm_workspace_size(c.mode, c.r, len(c.offsets) - 1, n, k, gather)
    buf = torch.full((size + GUARD,), 0xa5, dtype=torch.uint8, device="cuda")
    return buf[:size], buf[size:]


def on_pairs(c, n, k):
    """Whether the call runs on pairs of SMs: only there do gathered rows take space."""
    size = [fg.grouped_gemm_workspace_size(c.mode, c.r, len(c.offsets) - 1, n, k, gather) for gather in (False, True)]
    return size[1] > size[0]


@pytest.mark.parametrize("mode", ["mxfp8_b32", "mxfp4", "bf16", "fp8_block128"])
@pytest.mark.parametrize("total,n,experts", [(60, 256, 6), (4800, 512, 16)])
@pytest.mark.parametrize("gather", [True, False])
def test_offsets_that_decrease(mode, total, n, experts, gather):
    """An offset below an earlier one counts as the earlier one, and nothing is written past the workspace."""
    k = 512
    c = Experts(mode, [total // experts] * experts, n, k, total, gather_from=50 if gather else None)
    assert on_pairs(c, n, k) == (total == 4800 and mode != "fp8_block128")
    rng = np.random.default_rng(total)
    zigzag = [total * (e % 2) for e in range(experts + 1)]
    falls = sorted(rng.integers(0, total, experts + 1).tolist())
    falls[experts // 2] = 0
    falls[-1] = total // 2
    wild = rng.integers(-(1 << 31), (1 << 31) - 1, experts + 1).tolist()
    for offsets in (zigzag, falls, zigzag[::-1], wild):
        c.offsets = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        ws, guard = guarded(c, n, k, gather)
        y = torch.full((total, n), 3.0, dtype=torch.bfloat16, device="cuda")
        c.run(Y=y, workspace=ws)
        assert (guard == 0xa5).all(), offsets
        c.offsets = torch.from_numpy(np.maximum.accumulate(np.clip(offsets, 0, total)).astype(np.int32)).cuda()
        lo, hi = int(c.offsets[0]), int(c.offsets[-1])
        assert (y[:lo] == 3).all() and (y[hi:] == 3).all()
        if hi > lo:
            assert_close(y[lo:hi], c.reference()[lo:hi], offsets)


def words(ws, c, n, k):
    """The tickets of a 32-row call: the last of the workspace's (two 32 x 128 fp32 partials and a ticket) a block."""
    blocks = ws.numel() // (2 * 32 * 128 * 4 + 8)
    assert blocks * (2 * 32 * 128 * 4 + 8) == ws.numel()
    return ws[-8 * blocks:].view(torch.int64)


@pytest.mark.parametrize("mode", ["mxfp8_b32", "mxfp4_fp8a", "fp8_block128"])
def test_a_call_that_gave_up_leaves_no_arrivals(mode):
    """Shared units' tickets are clear after every call, also one that ran out of time: a replay of a captured call
    carries the call's tag and would count arrivals that an earlier run left."""
    n, k = 512, 4096
    c = Experts(mode, [3] * 8, n, k, 22)
    want = c.run()
    ws, guard = guarded(c, n, k, False)
    assert torch.equal(c.run(workspace=ws), want)
    shared = words(ws, c, n, k) == 0              # (the buffer held 0xa5 bytes)
    assert shared.any() and not shared.all()
    ws.fill_(0xa5)
    torch.cuda.synchronize()
    fg.set_wait_timeout_ns(20_000_000)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run(workspace=ws, flags=fg.FG_FLAG_DEBUG_STALL)
    finally:
        fg.set_wait_timeout_ns(4_000_000_000)
    for _ in range(2):
        graph.replay()
        assert fg.get_error() == fg.FG_ERR_TIMEOUT
        assert torch.equal(words(ws, c, n, k) == 0, shared)
    assert torch.equal(c.run(workspace=ws), want) and fg.get_error() == fg.FG_OK
    assert (guard == 0xa5).all()
