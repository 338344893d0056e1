"""Host-side checks of the microscaled entry points that need no GPU."""
import ctypes

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GemmEpiError, binding, build, mx_scales_bytes


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def test_scales_bytes(L):
    assert mx_scales_bytes(1, 32) == 512
    assert mx_scales_bytes(128, 128) == 512
    assert mx_scales_bytes(129, 160, batch=3) == 3 * 2 * 2 * 512
    # 5 groups of 300 rows: at most 300 / 128 whole tiles and one part each
    assert mx_scales_bytes(300, 128, groups=5) == (2 + 5) * 512
    assert mx_scales_bytes(3, 128, groups=5) == 3 * 512


@pytest.mark.parametrize("rows,cols,batch,groups", [(0, 32, 1, 0), (4, 33, 1, 0), (4, 0, 1, 0), (4, 32, 0, 0), (4, 32, 2, 3),
                                                    (4, 32, 1, 1025), (4, 32, 1, -1), (1 << 31, 32, 1, 0),
                                                    (1 << 30, 1 << 24, 1, 0)])
def test_bad_shapes(L, rows, cols, batch, groups):
    assert L.gemm_epi_mx_scales_bytes(batch, rows, cols, groups) == -1
    assert L.gemm_epi_mx_quantize(batch, rows, cols, 0, 0, 16, 16, groups, 16, 16, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_mx_dequantize(batch, rows, cols, 0, 0, 16, 16, 16, groups, 16, None) == binding.ERR_INVALID_ARG


def test_quantize_refusals(L):
    ok = (1, 64, 64, 0)
    assert L.gemm_epi_mx_quantize(*ok, 2, 16, None, 0, 16, 16, None) == binding.ERR_INVALID_ARG      # flags
    assert L.gemm_epi_mx_quantize(1, 64, 64, 5, 0, 16, None, 0, 16, 16, None) == binding.ERR_INVALID_ARG  # dtype
    assert L.gemm_epi_mx_quantize(*ok, 0, None, None, 0, 16, 16, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_mx_quantize(*ok, 0, 16, None, 2, 16, 16, None) == binding.ERR_INVALID_ARG      # no offsets
    assert L.gemm_epi_mx_quantize(*ok, 0, 24, None, 0, 16, 16, None) == binding.ERR_MISALIGNED
    assert L.gemm_epi_mx_quantize(*ok, 0, 16, 18, 2, 16, 16, None) == binding.ERR_MISALIGNED
    assert L.gemm_epi_mx_quantize(1, 60, 64, 0, 1, 16, None, 0, 16, 16, None) == binding.ERR_INVALID_ARG  # rows % 8
    assert L.gemm_epi_mx_quantize(1, 64, 64, 0, 1, 16, 16, 2, 16, 16, None) == binding.ERR_INVALID_ARG    # groups
    assert L.gemm_epi_mx_dequantize(*ok, 1, 16, 16, None, 0, 16, None) == binding.ERR_INVALID_ARG


@pytest.mark.parametrize("E,T,N,K,epi,flags,word", [(-1, 8, 64, 64, 0, 0, "experts"), (1025, 8, 64, 64, 0, 0, "experts"),
                                                    (0, 0, 64, 64, 0, 0, "shape"), (0, 8, 64, 48, 0, 0, "shape"),
                                                    (0, 8, 60, 64, 0, 0, "shape"), (0, 8, 64, 64, 2, 0, "epilog"),
                                                    (0, 8, 64, 64, 3, 0, "epilog"), (0, 8, 64, 64, 0, 1, "flags")])
def test_plan_refusals(L, E, T, N, K, epi, flags, word):
    assert not L.gemm_epi_mx_plan(E, T, N, K, 0, epi, flags)
    assert word in binding.gemm_epi_last_error()


def test_unknown_handle(L):
    assert L.gemm_epi_mx_execute(ctypes.c_void_p(0x1234), 16, 16, 16, 16, 16, None, 16, None) == binding.ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device error path")
def test_without_a_device(L):
    assert not L.gemm_epi_mx_plan(0, 64, 64, 64, 0, 0, 0)
    assert L.gemm_epi_mx_quantize(1, 64, 64, 0, 0, 16, None, 0, 16, 16, None) != 0
    with pytest.raises(GemmEpiError):
        binding.MxPlan(64, 64, 64, torch.bfloat16, "BIAS")
