"""Few-row gated plans and plans of 4-bit weights compute right results after a launch that gave up a wait.

One CTA of the first launch withholds its first completion signal: the parts of a tile that it shares with
others are counted in and its own is not. The plan's next calls bring other rows, other outputs and another
stream. Whole numbers, so sums are exact.
"""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GatedPlan, W4Plan, w4_pack

from test_recovery_gpu import BF, ints, recover, stall  # noqa: F401 (a fixture)
from test_w4_gpu import rowmajor, values, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("read_by_call", [False, True])
@pytest.mark.parametrize("T,gated,zeros", [(20, False, True), (20, True, False), (200, False, False)])
def test_four_bit_weights(stall, T, gated, zeros, read_by_call):  # noqa: F811
    N, K, G = 400, 2816, 64
    stall.setenv("GEMM_EPI_FORCE_KERNEL", "tmem")
    stall.setenv("GEMM_EPI_SKINNY_GRID", "19")
    codes, s, z = weights(N, K, G, BF, 4, zeros, True, 2 if gated else None)
    w4 = w4_pack(rowmajor(codes), s, z)
    Xs = ints((T, K), 3), ints((T, K), 1)
    Ys = torch.zeros((T, N), device="cuda"), torch.zeros((T, N), device="cuda")
    y = Xs[1].double() @ values(codes, s, z, G).reshape(-1, K).t()
    ref = (y[:, :N].clamp(min=0) * y[:, N:]).float() if gated else y.float()
    with W4Plan(T, N, K, BF, "GATED" if gated else "NONE", group=G, act="RELU", out_f32=True) as p:
        assert p.info()["split_k"] > 1 and p.info()["workspace_bytes"] > 0
        recover(p, lambda st, i: p.gemm_epi_w4_execute(Xs[i], *w4, None, Ys[i], stream=st),
                lambda: torch.equal(Ys[1], ref) or pytest.fail("Y"), read_by_call)


@pytest.mark.parametrize("read_by_call", [False, True])
@pytest.mark.parametrize("T,N,grid", [(20, 264, 11), (9, 9600, 70)])
@pytest.mark.parametrize("w_nk", [False, True])
def test_gated_layers(stall, T, N, grid, w_nk, read_by_call):  # noqa: F811
    K = 2048
    stall.setenv("GEMM_EPI_FORCE_KERNEL", "skinny")
    stall.setenv("GEMM_EPI_SKINNY_GRID", str(grid))
    W = ints((2 * N, K) if w_nk else (K, 2 * N), 2)
    Xs = ints((T, K), 3), ints((T, K), 1)
    Hs = torch.zeros((T, N), device="cuda"), torch.zeros((T, N), device="cuda")
    z = Xs[1].double() @ (W.double().t() if w_nk else W.double())
    ref = (z[:, :N].clamp(min=0) * z[:, N:]).float()
    with GatedPlan(T, N, K, BF, "GATED", act="RELU", w_nk=w_nk, out_f32=True) as p:
        assert p.info()["kernel"] == 1 and p.info()["split_k"] > 1
        recover(p, lambda st, i: p.gemm_epi_gated_execute(Xs[i], W, None, Hs[i], stream=st),
                lambda: torch.equal(Hs[1], ref) or pytest.fail("H"), read_by_call)
