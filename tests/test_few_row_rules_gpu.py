"""Which few-row kernel a plan takes, at shapes on either side of the stated rules (tile_m 32: each warp alone)."""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GatedPlan

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
