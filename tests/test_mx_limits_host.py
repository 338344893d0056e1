"""A microscaled plan takes no contraction whose scales the library cannot lay out."""
import pytest

from gemm_epilogues_tcgen05_b200 import binding, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def test_the_longest_row_is_the_same_everywhere(L):
    longest = 1 << 22
    assert L.gemm_epi_mx_scales_bytes(1, 8, longest, 0) == longest // 128 * 512
    for cols in (longest + 32, 1 << 23, 1 << 24):
        assert L.gemm_epi_mx_scales_bytes(1, 8, cols, 0) == -1
        assert "4194304" in binding.gemm_epi_last_error()
        assert not L.gemm_epi_mx_plan(0, 8, 64, cols, 0, 0, 0)
        assert "4194304" in binding.gemm_epi_last_error()
