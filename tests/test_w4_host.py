"""Host-side checks of the entry points for 4-bit weights with group scales that need no GPU."""
import ctypes

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GemmEpiError, W4Plan, binding, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def test_sizes(L):
    assert L.gemm_epi_w4_bytes(1, 32, 128, 128) == 2048 and L.gemm_epi_w4_scales(1, 32, 128, 128) == 32
    assert L.gemm_epi_w4_bytes(1, 33, 160, 32) == 4 * 2048 and L.gemm_epi_w4_scales(1, 33, 160, 32) == 4 * 128
    assert L.gemm_epi_w4_bytes(3, 1, 64, 64) == 3 * 2048 and L.gemm_epi_w4_scales(3, 1, 64, 64) == 3 * 64


@pytest.mark.parametrize("batch,rows,cols,group", [(1, 16, 128, 16), (1, 16, 128, 0), (1, 16, 96, 64), (1, 0, 128, 64), (0, 16, 128, 64),
                                                   (1, 16, 0, 32), (1, 16, -128, 128), (1, 1 << 25, 128, 128),
                                                   (1, 16, 1 << 23, 128), (1 << 20, 1 << 24, 1 << 22, 128)])
def test_bad_shapes(L, batch, rows, cols, group):
    shape = (batch, rows, cols, group)
    assert L.gemm_epi_w4_bytes(*shape) == -1 and L.gemm_epi_w4_scales(*shape) == -1
    assert binding.gemm_epi_last_error()
    assert L.gemm_epi_w4_quantize(*shape, 0, 32, 32, 32, None, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_w4_pack(*shape, 32, 32, None, 32, 32, None, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_w4_dequantize(*shape, 0, 0, 32, 32, None, 32, None) == binding.ERR_INVALID_ARG


def test_refusals(L):
    ok = (1, 64, 256, 64)
    assert L.gemm_epi_w4_quantize(*ok, 5, 32, 32, 32, None, None) == binding.ERR_INVALID_ARG   # dtype
    assert L.gemm_epi_w4_quantize(*ok, 0, None, 32, 32, None, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_w4_quantize(*ok, 0, 32, 40, 32, None, None) == binding.ERR_MISALIGNED
    assert L.gemm_epi_w4_quantize(*ok, 0, 32, 32, 32, 8, None) == binding.ERR_MISALIGNED
    assert L.gemm_epi_w4_pack(*ok, 32, 32, 32, 32, 32, None, None) == binding.ERR_INVALID_ARG  # zeros on one side
    assert L.gemm_epi_w4_pack(*ok, 32, 32, None, 32, 32, 32, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_w4_pack(*ok, 32, 33, None, 32, 32, None, None) == binding.ERR_MISALIGNED
    assert L.gemm_epi_w4_dequantize(*ok, 0, 1, 32, 32, None, 32, None) == binding.ERR_INVALID_ARG  # flags
    assert L.gemm_epi_w4_dequantize(*ok, 0, 0, 32, None, None, 32, None) == binding.ERR_INVALID_ARG
    assert L.gemm_epi_w4_dequantize(*ok, 0, 0, 24, 32, None, 32, None) == binding.ERR_MISALIGNED


@pytest.mark.parametrize("T,N,K,group,dtype,epi,act,flags,word",
                         [(0, 64, 256, 64, 0, 0, 0, 0, "shape"), (257, 64, 256, 64, 0, 0, 0, 0, "dequantize"),
                          (4, 60, 256, 64, 0, 0, 0, 0, "shape"), (4, 64, 256, 48, 0, 0, 0, 0, "group"),
                          (4, 64, 96, 64, 0, 0, 0, 0, "shape"), (4, 64, 256, 64, 3, 0, 0, 0, "dtype"),
                          (4, 64, 256, 64, 0, 2, 0, 0, "epilog"), (4, 64, 256, 64, 0, 9, 0, 0, "epilog"),
                          (4, 64, 256, 64, 0, 10, 0, 0, "epilog"), (4, 64, 256, 64, 0, 8, 7, 0, "activation"),
                          (4, 64, 256, 64, 0, 0, 0, 1, "flags")])
def test_plan_refusals(L, T, N, K, group, dtype, epi, act, flags, word):
    assert not L.gemm_epi_w4_plan(T, N, K, group, dtype, epi, act, flags)
    assert word in binding.gemm_epi_last_error()


def test_unknown_handle(L):
    assert L.gemm_epi_w4_execute(ctypes.c_void_p(0x1234), 32, 32, 32, None, None, 32, None) == binding.ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device error path")
def test_without_a_device(L):
    assert not L.gemm_epi_w4_plan(4, 64, 256, 64, 0, 0, 0, 0)
    assert L.gemm_epi_w4_quantize(1, 64, 256, 64, 0, 32, 32, 32, None, None) != 0
    with pytest.raises(GemmEpiError):
        W4Plan(4, 64, 256, torch.bfloat16, "NONE")
    with pytest.raises(ValueError):
        binding.gemm_epi_w4_quantize(torch.zeros(64, 256, dtype=torch.bfloat16), None, None)
