"""Which few-row kernel a plan takes, at shapes on either side of the stated rules (tile_m 32: each warp alone)."""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GatedPlan, W4Plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,alone", [(2048, 1024, True), (2048, 2048, True), (1024, 3008, True), (2048, 3584, True),
                                       (4096, 2048, True), (1024, 4096, False), (1536, 4096, False), (2048, 4096, False),
                                       (2360, 4096, False), (512, 4096, False), (256, 8192, False), (5632, 1024, False),
                                       (3000, 3000, False), (11008, 4096, False)])
@pytest.mark.parametrize("T", [1, 16])
def test_gated_layers(N, K, alone, T):
    with GatedPlan(T, N, K, torch.bfloat16) as p:
        info = p.info()
        assert info["kernel"] == 1 and (info["tile_m"] == 32) == alone
        assert not alone or info["split_k"] == 1


@pytest.mark.parametrize("T,N,K,gated,alone", [(1, 128000, 4096, False, True), (16, 11008, 4096, False, True), (32, 4096, 4096, False, True),
                                               (64, 4096, 4096, True, True), (48, 5000, 2048, False, True), (32, 11008, 4096, True, True),
                                               (17, 11008, 4096, False, False), (32, 11008, 4096, False, False),
                                               (64, 11008, 2048, False, False), (48, 11008, 4096, True, False), (128, 11008, 4096, True, False)])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_four_bit_weights(T, N, K, gated, alone, G):
    with W4Plan(T, N, K, torch.bfloat16, "GATED" if gated else "NONE", group=G) as p:
        assert p.info()["tile_m"] == (32 if alone else 128)
