"""Host-side checks of the gated-layer entry points that need no GPU: refusals
come before any device call, with a message."""
import ctypes

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GatedPlan, GemmEpiError, binding, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


@pytest.mark.parametrize("T,N,K", [(0, 64, 64), (-1, 64, 64), (8, 0, 64), (8, 12, 64), (8, 64, 4), (8, 64, 100),
                                   (1 << 31, 64, 64), (8, 1 << 24, 64), (1 << 30, 1 << 20, 64), (1 << 30, 1 << 14, 64)])
def test_plan_rejects_bad_shapes(L, T, N, K):
    assert not L.gemm_epi_gated_plan(T, N, K, 0, 8, 0, 0)
    assert "shape" in binding.gemm_epi_last_error()


@pytest.mark.parametrize("dtype,epilog,act,flags,word", [(7, 8, 0, 0, "dtype"), (0, 0, 0, 0, "epilog"), (0, 7, 0, 0, "epilog"),
                                                         (0, 11, 0, 0, "epilog"), (0, 8, 3, 0, "activation"),
                                                         (0, 9, -1, 0, "activation"), (0, 8, 0, 4, "flags")])
def test_plan_rejects_bad_enums_and_flags(L, dtype, epilog, act, flags, word):
    assert not L.gemm_epi_gated_plan(64, 64, 64, dtype, epilog, act, flags)
    assert word in binding.gemm_epi_last_error()


def test_other_plans_have_no_gated_epilog(L):
    for epilog in binding.GATED_EPILOGS.values():
        assert not L.gemm_epi_plan(64, 64, 64, 0, epilog)
        assert not L.gemm_epi_grouped_plan(2, 64, 64, 64, 0, epilog, 0)
        assert not L.gemm_epi_mx_plan(0, 64, 64, 64, 0, epilog, 0)


def test_unknown_handles_are_rejected(L):
    bogus = ctypes.c_void_p(0x12345678)
    assert L.gemm_epi_gated_execute(bogus, 16, 16, 16, 16, 16, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_dgated_execute(bogus, 16, 16, 16, 16, 16, None) == binding.ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device error path")
def test_plan_without_a_device_fails_cleanly(L):
    assert not L.gemm_epi_gated_plan(256, 256, 256, 0, 8, 0, 0)
    assert binding.gemm_epi_last_error()
    with pytest.raises(GemmEpiError):
        GatedPlan(256, 256, 256, torch.bfloat16)
