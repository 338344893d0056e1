"""Zero points that 7 bits do not hold: a group of one stands for NaN, its neighbours for what they are."""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import W4Plan, gemm_epi_w4_dequantize, w4_pack

from test_w4_gpu import DT, ints, gen, rowmajor, values, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,G", [(8, 32, 32), (40, 192, 64), (72, 384, 32), (264, 1152, 128)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_a_group_of_a_large_zero_point_is_nan(N, K, G, dt):
    dt = DT[dt]
    codes, s, z = weights(N, K, G, dt, N, True, True)
    z[:, 0] = 127
    z[3, -1], z[N - 1, 0], z[5, 0] = 128, 255, 200
    q, ps, pz = w4_pack(rowmajor(codes), s, z)
    bad = (z > 127)[..., None].expand(N, K // G, G).reshape(N, K)
    ref = values(codes, s, z, G)
    for out in (torch.empty((N, K), device="cuda"), torch.empty((N, K), dtype=dt, device="cuda")):
        gemm_epi_w4_dequantize(q, ps, pz, out, group=G)
        assert torch.equal(out.isnan(), bad)
        assert torch.equal(out[~bad], ref.float().to(out.dtype)[~bad])
    for T in (1, 12, 200):
        X = ints((T, K), 3, gen(T), dt)
        with W4Plan(T, N, K, dt, "NONE", group=G, out_f32=True) as p:
            Y = p.forward(X, q, ps, pz)
        rows = bad.any(1)
        assert bool(Y[:, rows].isnan().all())
        assert torch.equal(Y[:, ~rows].double(), X.double() @ ref[~rows].t())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_a_byte_laid_out_by_hand_shows_as_nan(dt):
    dt = DT[dt]
    codes, s, z = weights(32, 128, 128, dt, 1, True, True)
    q, ps, pz = w4_pack(rowmajor(codes), s, z)
    pz[7] = 131
    for out in (torch.empty((32, 128), device="cuda"), torch.empty((32, 128), dtype=dt, device="cuda")):
        gemm_epi_w4_dequantize(q, ps, pz, out, group=128)
        assert bool(out[7].isnan().all()) and int(out.isnan().sum()) == 128
