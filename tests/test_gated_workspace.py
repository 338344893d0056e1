"""The bias gradient's workspace of a DGATED plan is the caller's choice."""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GatedPlan, GemmEpiError, binding, build

NO_DBIAS = 4


def test_the_flag_belongs_to_dgated_plans():
    build.build()
    L = binding.lib()
    for epilog in ("GATED", "GATED_AUX"):
        assert not L.gemm_epi_gated_plan(64, 64, 64, 0, binding.GATED_EPILOGS[epilog], 0, NO_DBIAS)
        assert "flags" in binding.gemm_epi_last_error()
    assert not L.gemm_epi_gated_plan(64, 64, 64, 0, binding.GATED_EPILOGS["DGATED"], 0, NO_DBIAS | 8)
    assert "flags" in binding.gemm_epi_last_error()
    assert not L.gemm_epi_plan_ex(64, 64, 64, 0, 3, NO_DBIAS)
    assert "flags" in binding.gemm_epi_last_error()


@pytest.mark.gpu
def test_without_a_bias_gradient_there_is_no_workspace():
    T, N, K, bf = 300, 264, 136, torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dY, W2, Z = (torch.randn(s, generator=g, device="cuda").to(bf) for s in ((T, K), (K, N), (T, 2 * N)))
    dbias = torch.full((2 * N,), 77.0, device="cuda")
    with GatedPlan(T, N, K, bf, "DGATED") as p, GatedPlan(T, N, K, bf, "DGATED", dbias=False) as q:
        assert p.info()["workspace_bytes"] >= 10 * 2 * N * 4 and q.info()["workspace_bytes"] == 0
        a, b = p.backward(dY, W2, Z), q.backward(dY, W2, Z)
        assert torch.equal(a, b)
        b.fill_(77)
        with pytest.raises(GemmEpiError, match="NO_DBIAS") as e:
            q.gemm_epi_dgated_execute(dY, W2, Z, b, dbias)
        assert e.value.code == binding.ERR_INVALID_ARG
        torch.cuda.synchronize()
        assert bool((b == 77).all()) and bool((dbias == 77).all())  # nothing ran
        assert torch.equal(q.backward(dY, W2, Z), a) and q.status() == 0


@pytest.mark.gpu
def test_a_long_batch_takes_no_memory():
    torch.zeros(1, device="cuda")
    T, N, K = 65536, 28672, 64
    with GatedPlan(T, N, K, torch.bfloat16, "DGATED", dbias=False):
        pass  # (the kernel's module is loaded)
    before = torch.cuda.mem_get_info()[0]
    with GatedPlan(T, N, K, torch.bfloat16, "DGATED", dbias=False):
        assert before - torch.cuda.mem_get_info()[0] < 16 << 20
