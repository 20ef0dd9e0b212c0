"""Workspace sizes of the grouped product in fp8_block128, which has two forms."""
import pytest

import mx_gemm_gb300 as fg


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("experts,n,k", [(1, 128, 128), (4, 128, 7168), (8, 256, 1024), (16, 384, 2048), (64, 128, 4096), (64, 4096, 7168)])
def test_what_is_enough_is_enough_for_fewer_rows(experts, n, k, gather):
    last = 0
    for rows in list(range(1, 300)) + list(range(300, 40000, 97)):
        size = fg.grouped_gemm_workspace_size("fp8_block128", rows, experts, n, k, gather)
        assert size >= last, rows
        last = size
    assert not gather or last >= rows * k
