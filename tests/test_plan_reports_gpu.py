"""What plans report: errors that stay with their call."""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GemmEpiError, GroupedPlan, Plan

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
