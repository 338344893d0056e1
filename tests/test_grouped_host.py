"""Host-side checks of the expert-grouped entry points that need no GPU:
refusals come before any device call, with a message."""
import ctypes

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import binding, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


@pytest.mark.parametrize("E,T,N,K,word", [(0, 8, 64, 64, "experts"), (1025, 8, 64, 64, "experts"), (-1, 8, 64, 64, "experts"),
                                          (4, 0, 64, 64, "shape"), (4, 8, 12, 64, "shape"), (4, 8, 64, 100, "shape"),
                                          (4, 8, 0, 64, "shape"), (4, 1 << 31, 64, 64, "shape"),
                                          (1024, 1 << 30, 1 << 11, 64, "shape"), (2, 8, 1 << 24, 1 << 14, "shape")])
def test_plan_rejects_bad_shapes(L, E, T, N, K, word):
    assert not L.gemm_epi_grouped_plan(E, T, N, K, 0, 0, 0)
    assert word in binding.gemm_epi_last_error()


def test_plan_rejects_bad_enums_and_flags(L):
    assert not L.gemm_epi_grouped_plan(2, 64, 64, 64, 7, 0, 0)
    assert "dtype" in binding.gemm_epi_last_error()
    assert not L.gemm_epi_grouped_plan(2, 64, 64, 64, 0, 8, 0)
    assert "epilog" in binding.gemm_epi_last_error()
    assert not L.gemm_epi_grouped_plan(2, 64, 64, 64, 0, 0, 4)
    assert "flags" in binding.gemm_epi_last_error()
    assert not L.gemm_epi_grouped_plan(2, 64, 64, 64, 0, binding.WGRAD, binding.FLAG_W_NK)
    assert "W_NK" in binding.gemm_epi_last_error()


def test_unknown_handles_are_rejected(L):
    bogus = ctypes.c_void_p(0x12345678)
    assert L.gemm_epi_grouped_execute(bogus, 16, 16, 16, 16, 16, 16, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_grouped_drelu_bgrad_execute(bogus, 16, 16, 16, 16, 16, 16, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_grouped_wgrad_execute(bogus, 16, 16, 16, 16, 16, None) == binding.ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device error path")
def test_plan_without_a_device_fails_cleanly(L):
    assert not L.gemm_epi_grouped_plan(4, 256, 256, 256, 0, 2, 0)
    assert binding.gemm_epi_last_error()
    with pytest.raises(binding.GemmEpiError):
        binding.GroupedPlan(4, 256, 256, 256, torch.bfloat16, "BIAS")
