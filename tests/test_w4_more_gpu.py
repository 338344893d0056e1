"""4-bit weights: batches, prompts of a gated layer, offsets beyond 32 bits."""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GatedPlan, GemmEpiError, W4Plan, gemm_epi_w4_dequantize, w4_pack, w4_quantize

from test_gated_gpu import E, TINY, U, act, gen, ints, within
from test_w4_gpu import DT, reference_codes, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,K,G", [(2, 1, 32, 32), (3, 40, 192, 64), (5, 33, 416, 32), (2, 100, 1152, 128)])
@pytest.mark.parametrize("zeros", [False, True])
def test_batches_of_ragged_matrices(B, N, K, G, zeros):
    dt = torch.bfloat16
    W = (torch.randn((B, N, K), generator=gen(N), device="cuda") / 8).to(dt)
    q, s, z = w4_quantize(W, group=G, zeros=zeros)
    ref = []
    for m in range(B):
        c, rs, rz = reference_codes(W[m], G, zeros)
        ref.append(values(c, rs, rz if zeros else None, G))
        alone = w4_quantize(W[m].contiguous(), group=G, zeros=zeros)
        for whole, part in zip((q, s, z), alone):  # whole tiles, one matrix after the other
            assert whole is None or torch.equal(whole.view(B, -1)[m], part)
    ref = torch.stack(ref)
    out = torch.empty((B, N, K), device="cuda")
    gemm_epi_w4_dequantize(q, s, z, out, group=G)
    assert torch.equal(out.double(), ref)
    out16 = torch.empty((B, N, K), dtype=dt, device="cuda")
    gemm_epi_w4_dequantize(q, s, z, out16, group=G)
    assert torch.equal(out16, ref.float().to(dt))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["SILU", "GELU", "RELU"])
def test_gated_prompt_through_the_same_weight(name, dt):
    """More rows than the plan takes: both matrices dequantised to 16 bits are the 2N x K weight of a gated plan. That
    and the 4-bit plan's rows of the same prompt against 64 bits, each with its own weight: sums of K products err
    by 2 K e of their magnitudes (for 4 bits (256 + K / G + 8) e), |act'| <= 1.13, then the epilogue's errors."""
    T, N, K, G = 300, 264, 512, 64
    dt = DT[dt]
    W = (torch.randn((2, N, K), generator=gen(1), device="cuda") / 16).to(dt)
    q, s, z = w4_quantize(W, group=G, zeros=True)
    held, full = torch.empty_like(W), torch.empty((2, N, K), device="cuda")
    gemm_epi_w4_dequantize(q, s, z, held, group=G)
    gemm_epi_w4_dequantize(q, s, z, full, group=G)
    X = torch.randn((T, K), generator=gen(2), device="cuda").to(dt)
    with pytest.raises(GemmEpiError, match="dequantize"):
        W4Plan(T, N, K, dt, "GATED", group=G, act=name)
    with GatedPlan(T, N, K, dt, act=name, w_nk=True) as d, W4Plan(5, N, K, dt, "GATED", group=G, act=name) as p:
        H, _ = d.forward(X, held.view(2 * N, K))
        few = p.forward(X[100:105].contiguous(), q, s, z)
    for got, x, w, terms in ((H, X, held, 2 * K), (few, X[100:105], full, 2 * 128 + K / G + 8)):
        w = w.view(2 * N, K).double()
        y, err = x.double() @ w.t(), terms * E * (x.double().abs() @ w.abs().t())
        g, up, eg, eu = y[:, :N], y[:, N:], err[:, :N], err[:, N:]
        a, _, ea, _ = act(g, name)
        bound = (1.13 * eg + 2 * ea) * (up.abs() + 2 * eu) + eu * a.abs()
        u = U[dt]
        within(got, a * up, (1 + u) * bound + (u + 2 * E) * (a * up).abs() + TINY[dt], name)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("kernel,T", [("warp", 2), ("tmem", 20)])
def test_codes_beyond_32_bit_offsets(kernel, T, zeros, monkeypatch):
    """4.6 GB of codes; rows at the beginning, around 2^31 and 2^32 bytes, and the last ones."""
    monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", kernel)
    N, K, G, dt = 2200000, 4160, 32, torch.bfloat16
    g = gen(1)
    packed = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (2.0 ** torch.randint(-6, -3, (N, K // G), generator=g, device="cuda", dtype=torch.int8).float()).to(dt)
    z = torch.randint(0, 16, (N, K // G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    w4 = w4_pack(packed, s, z)
    per_row = w4[0].numel() // ((N + 31) // 32) // 32
    at = [0, 1, 2 ** 31 // per_row - 1, 2 ** 31 // per_row + 33, 2 ** 32 // per_row - 40, 2 ** 32 // per_row + 1, 2 ** 32 // per_row + 70, N - 2, N - 1]
    assert w4[0].numel() > 2 ** 32
    X = ints((T, K), 2, gen(3), dt)
    with W4Plan(T, N, K, dt, "NONE", group=G, out_f32=True) as p:
        Y = p.forward(X, *w4)
        assert p.status() == 0
    rows = torch.tensor(at, device="cuda")
    codes = torch.stack([packed[rows] & 15, packed[rows] >> 4], -1).view(len(at), K)
    ref = X.double() @ values(codes, s[rows], None if z is None else z[rows], G).t()
    assert torch.equal(Y[:, rows].double(), ref)
    del Y, packed
    out = torch.empty((N, K), dtype=dt, device="cuda")
    gemm_epi_w4_dequantize(*w4, out, group=G)
    assert torch.equal(out[rows].double(), values(codes, s[rows], None if z is None else z[rows], G))
    if kernel == "warp" and not zeros:  # and a weight of more than 2^33 elements quantised: what comes back is a fixed point
        q2, s2, _ = w4_quantize(out, group=G)
        del w4
        last = slice(N - 64, N)
        c, rs, _ = reference_codes(out[last].contiguous(), G, False)
        back = torch.empty_like(out)
        gemm_epi_w4_dequantize(q2, s2, None, back, group=G)
        assert torch.equal(back[last].double(), values(c, rs, None, G).float().to(dt).double())
