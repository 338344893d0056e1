"""What plans report: the kernel's choices, and errors that stay with their call."""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GemmEpiError, GroupedPlan, MxPlan, Plan

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_an_allocation_that_fails_does_not_fail_the_next_call(monkeypatch):
    """A bias-gradient workspace of 206 GB is refused; the one-product launch after it is not."""
    X, W = torch.ones((200, 64), dtype=BF, device="cuda"), torch.ones((64, 72), dtype=BF, device="cuda")
    b = torch.zeros(72, dtype=BF, device="cuda")
    with Plan(200, 72, 64, BF, "BIAS") as p:
        assert p.info()["kernel"] == 0
        monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", "32")
        with pytest.raises(GemmEpiError, match="workspace"):
            GroupedPlan(1024, 1 << 16, 1 << 24, 8, BF, "DRELU_BGRAD")
        Y, _ = p.forward(X, W, b)
        torch.cuda.synchronize()
        assert bool((Y == 64).all())


def test_split_and_launches(monkeypatch):
    """split_k: the CTAs that share a tile of the mean expert's rows; 1 where none can."""
    # one narrow expert over a long contraction, and the weight gradient of many rows
    with GroupedPlan(1, 5, 64, 4096, BF, "DRELU_BGRAD") as p, GroupedPlan(1, 8192, 64, 64, BF, "WGRAD") as w:
        assert 2 <= p.info()["split_k"] <= 16 and 2 <= w.info()["split_k"] <= 16
        assert p.info()["workspace_bytes"] > 0 and p.info()["launches"] == 1 and w.info()["launches"] == 1
    with GroupedPlan(8, 8192, 4096, 4096, BF, "BIAS") as p, MxPlan(4, 512, 8192, BF, "BIAS") as m:
        assert p.info()["split_k"] == 1 and m.info()["split_k"] == 1 and m.info()["launches"] == 1
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", "32")
    for want in (1, 3, 16):
        monkeypatch.setenv("GEMM_EPI_FORCE_SPLIT", str(want))
        with GroupedPlan(1, 5, 64, 4096, BF, "BIAS") as p:
            assert p.info()["split_k"] == want
    monkeypatch.setenv("GEMM_EPI_FORCE_SPLIT", "16")
    with GroupedPlan(64, 64, 512, 4096, BF, "BIAS") as p:  # 256 tiles: no room to share
        assert p.info()["split_k"] == 1
