"""The stored ncu traffic figure belongs to the GEMM's kernels: it outlives
edits of the operators around the GEMM, and not edits of its own sources."""
import os

import pytest

import bench
import mx_gemm_gb300 as fg
from tests.test_bench_host import _digest_of

CSRC = os.path.join(os.path.dirname(fg.__file__), "csrc")


def test_the_default_workload_has_a_figure_for_these_kernels():
    assert bench.traffic(bench.DEFAULT_WORKLOAD, fg) is not None


def test_sources_are_followed_through_their_includes():
    names = bench.gemm_sources(CSRC)
    assert set(bench.GEMM_UNITS) <= set(names) and {"fg_ptx.cuh", "fg_internal.cuh", "fg_tiles.cuh"} <= set(names)
    assert not {"fg_moe.cu", "fg_quant.cu", "fg_grouped.cu", "fg_grouped.cuh"} & set(names)


@pytest.mark.parametrize("edit", [("fg_moe.cu", "constexpr int kGroup = 64;", "constexpr int kGroup = 32;"),
                                  ("fg_quant.cu", "constexpr int kVec = 8;", "constexpr int kVec = 4;"),
                                  ("fg_grouped.cuh", "constexpr int kMaxExperts = 1024;", "constexpr int kMaxExperts = 512;")])
def test_other_operators_do_not_matter(tmp_path, edit):
    assert _digest_of(tmp_path, edit) == bench.kernel_sources_digest(fg)


@pytest.mark.parametrize("edit", [("fg_api.cu", "{FG_FP8_TENSOR, 1, 16384, 7168, 2, 2, 3}", "{FG_FP8_TENSOR, 1, 16384, 7168, 1, 2, 3}"),
                                  ("fg_tiles.cuh", "return", "return  1 +")])
def test_the_gemm_does(tmp_path, edit):
    assert _digest_of(tmp_path, edit) != bench.kernel_sources_digest(fg)
