"""GELU of the grouped and microscaled products over its whole range.

With W = 0 and an fp32 bias the pre-activation is the bias itself, any fp32
number. gelu(z) = max(z, 0) - |z| h(|z|) with h(a) = Phi(-a) = 2^q(a), q(a) =
-1 + a (s(a) - a / (2 ln 2)), s a polynomial. In steps of e = 2^-24 (half a
unit in the last place, relative):
  * s is below 1.2 in magnitude and off by at most 2 e of its fit and 3 e of
    its evaluation (1 e the last rounding, 0.75 e the argument's, the rest the
    roundings before and of the coefficients): a s is off by 5 e a;
  * s - a / (2 ln 2) is one rounding and a (s - ...) = q + 1: e (|q| + 1); its
    constant is off by e / 4: less than e |q| / 2;
  * the last one rounds q: e |q|. In all |dq| <= (2.5 |q| + 1 + 5 a) e, which
    moves 2^q by ln 2 of it, relatively;
  * the exponential function: 2^-22 = 4 e;
  * one rounding of the result: e |gelu|.
So |error| <= (ln 2 (2.5 |q| + 1 + 5 a) + 4) e |z| h + e |gelu|, and a rounding to
16 bits adds half a step of the result. h below 2^-126 becomes 0, which
happens below z = -12.9: there |gelu| is under 1.6e-37.
"""
import math

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GroupedPlan, MxPlan

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half of the least subnormal (bf16: far below 1.6e-37 is fine)


def sweep():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dense = torch.linspace(-14, 8, 1 << 19, device="cuda")
    near = torch.exp(torch.rand(1 << 16, generator=g, device="cuda") * 60 - 58)  # down to 6e-26
    far = torch.tensor([13.0, -13.0, -12.75, -12.99, -20.0, 50.0, -60000.0, 3e38, -3e38, 0.0, -0.0, 5.25, -5.25] + [0.0] * 3,
                       device="cuda")
    z = torch.cat([dense, near, -near, far])
    return torch.cat([z, z.new_zeros(-len(z) % 64)])


def reference(z):
    d = z.double()
    return d * torch.exp(torch.special.log_ndtr(d))


def allowed(z, ref):
    a = z.double().abs()
    q = torch.special.log_ndtr(-a) / math.log(2)
    h = torch.exp(torch.special.log_ndtr(-a))
    return (math.log(2) * (2.5 * q.abs() + 1 + 5 * a) + 4) * E24 * a * h + E24 * ref.abs() + 1.6e-37


def outputs(z, dt, out_f32):
    """GELU of z by each kernel that computes one: name -> values."""
    N, K = len(z), 32
    bias = z.float().contiguous()
    got = {}
    X, W = torch.ones((2, 32), dtype=dt, device="cuda"), torch.zeros((1, K, N), dtype=dt, device="cuda")
    offsets = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    for epilog in ("GELU_BIAS", "GELU_AUX_BIAS"):
        with GroupedPlan(1, 2, N, K, dt, epilog, out_f32=out_f32) as p:
            p.set_bias_f32()
            got[epilog] = p.forward(X, W, bias[None], offsets)[0]
    with MxPlan(2, N, K, dt, "GELU_BIAS", out_f32=out_f32) as p:
        p.set_bias_f32()
        zq, zs = torch.zeros((2, K // 2), dtype=torch.uint8, device="cuda"), torch.zeros(p.x_scales, dtype=torch.uint8, device="cuda")
        wq, ws = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda"), torch.zeros(p.w_scales, dtype=torch.uint8, device="cuda")
        got["microscaled"] = p.forward(zq, zs, wq, ws, bias)
    return got


@pytest.mark.parametrize("tr", [32, 128, 256])
def test_fp32_output_keeps_relative_accuracy(monkeypatch, tr):
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    z = sweep()
    ref = reference(z)
    bound = allowed(z, ref)
    for name, Y in outputs(z, torch.bfloat16, True).items():
        assert torch.equal(Y[0], Y[1]), name
        bad = (Y[0].double() - ref).abs() > bound
        assert not bool(bad.any()), (name, z[bad][:4].tolist(), Y[0][bad][:4].tolist(), ref[bad][:4].tolist())
        assert bool((Y[0][z < 0] <= 0).all()) and bool((Y[0][z > 0] >= 0).all()), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_16_bit_output_is_off_by_little_more_than_half_a_step(dtype):
    z = sweep()
    z = torch.where(z.abs() < 6e4, z, 0.0)
    ref = reference(z)
    own = allowed(z, ref)
    bound = own + STEP[dtype] * (ref.abs() + own) + LEAST[dtype]
    for name, Y in outputs(z, dtype, False).items():
        bad = (Y[0].double() - ref).abs() > bound
        assert not bool(bad.any()), (name, z[bad][:4].tolist(), Y[0][bad][:4].tolist(), ref[bad][:4].tolist())
        assert bool((Y[0][z < 0] <= 0).all()), name


def test_infinities_and_nan():
    z = torch.tensor([float("inf"), float("-inf"), float("nan")] + [1.0] * 5, device="cuda").repeat(8)
    for name, Y in outputs(z, torch.bfloat16, True).items():
        y = Y[0].view(8, 8)
        assert bool((y[:, 0] == float("inf")).all()) and bool((y[:, 1] == 0).all()) and bool(torch.isnan(y[:, 2]).all()), name
