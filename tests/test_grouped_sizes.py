"""Workspace sizes of the grouped product in fp8_block128, which has two forms."""
import pytest

import mx_gemm_gb300 as fg


@pytest.mark.parametrize("experts,n,k", [(1, 128, 128), (4, 128, 7168), (8, 256, 1024), (16, 384, 2048), (64, 128, 4096), (64, 4096, 7168)])
def test_sizes_without_gathering_never_fall(experts, n, k):
    last = 0
    for rows in list(range(1, 300)) + list(range(300, 40000, 97)):
        size, gathered = (fg.grouped_gemm_workspace_size("fp8_block128", rows, experts, n, k, g) for g in (False, True))
        assert size >= last and gathered in (size, max(size, rows * k)), rows
        last = size
