"""Sizes whose products leave 64 bits are refused like any other size that is
too large (no GPU needed)."""
import ctypes

import pytest

from tests.test_abi import fg  # noqa: F401  (fixture)
from tests.test_moe_abi import route


@pytest.mark.parametrize("T,k", [(1 << 59, 32), ((1 << 60) + 1, 16), ((1 << 62) + 4, 4), ((1 << 63) - 1, 2), ((1 << 30) // 8 + 1, 8)])
def test_route_tokens_times_choices(fg, T, k):  # noqa: F811
    """T * top_k must not pass for a small number of pairs."""
    assert route(fg, T=T, k=k, bytes=1 << 40) == fg.FG_ERR_SHAPE
    assert "fg_moe_route" in fg.last_error_message()


@pytest.mark.parametrize("N,E", [((1 << 54) + 128, 1024), (1 << 62, 4), ((1 << 61) + 128, 8), ((1 << 63) - 128, 1024)])
def test_grouped_rows_of_all_experts(fg, N, E):  # noqa: F811
    b = ctypes.c_uint64(7)
    assert fg.lib().fg_grouped_gemm_workspace_size(5, 8, E, N, 256, 0, ctypes.byref(b)) == fg.FG_ERR_SHAPE
    assert b.value == 7


@pytest.mark.parametrize("T", [(1 << 63) - 1, (1 << 63) - 64, (1 << 30) + 1])
def test_route_workspace_of_too_many_tokens(fg, T):  # noqa: F811
    b = ctypes.c_uint64(7)
    assert fg.lib().fg_moe_route_workspace_size(T, 64, ctypes.byref(b)) == fg.FG_ERR_SHAPE
    assert b.value == 7
