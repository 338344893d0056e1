"""Activations of gated layers and their derivatives over every 16-bit gate, relative to the value.

dH = U = 1, so that dG is act'(G) and dU is act(G), both fp32. Bounds in units of e = 2^-24, to
first order (a hundredth is added for the rest), of what the kernels evaluate:

SILU. E = e^-z by ex2 of a rounded product: ex2 errs by 2 ulp (4 e), the product's rounding and
  log2 e's own by 1.22 e of an exponent |z| log2 e, so r_E = (4 + 1.22 |z|) e. p = 1 / (1 + E): E's part
  of the sum is 1 - p, the sum's rounding e, the reciprocal 1 ulp (2 e): r_p = (1 - p) r_E + 3 e.
  a = z p: r_a = r_p + e. d = p + a (1 - p) in one multiply-add, 1 - p off by r_p p + e (1 - p):
  |a| (1 - p) (r_a + e) + |a| p r_p + r_p p + e |d|. From z = 18 on E is below 2^-25 and the sum is 1, so are p
  and d, which miss e^-z and (1 + z) e^-z.
  Below -88.72, where e^-z leaves fp32, p is 0: a and d miss |z| e^z <= 2.7e-37.
GELU. h = Phi(-|z|): r_h = 8e-7 to |z| = 4, 2e-6 to 6, 9e-6 to 12.9 (its stated errors), 0 beyond (2.2e-38
  at most). a = max(z, 0) - |z| h: |z| h r_h + e |a|. phi: the exponent's constant and two
  products 2.2 e of z^2 / 2, ex2 4 e, its factor and the product 2 e: r_phi = (6 + 1.1 z^2) e.
  d = z phi + Phi(z): |z| phi r_phi + h r_h + e (z > 0: 1 - h is rounded) + e |d|; below -12.9
  phi's flush counts 13.3 x 1.2e-38 too.
RELU. Exact.
"""
import math

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GatedPlan

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E = 2.0 ** -24


def bounds(z, name):
    """act(z), act'(z) and the bounds of their errors, in 64 bits."""
    if name == "SILU":
        p, q = torch.special.expit(z), torch.special.expit(-z)
        a = z * p
        d = p + a * q
        r_e = (4 + 1.22 * z.abs()) * E
        r_p = q * r_e + 3 * E
        r_a = r_p + E
        ea = r_a * a.abs()
        ed = a.abs() * q * (r_a + E) + a.abs() * p * r_p + r_p * p + E * d.abs()
        far = z >= 18
        ea, ed = torch.where(far, 2 * E * a.abs(), ea), torch.where(far, (1 + z.abs()) * q + E, ed)
        cut = torch.where(z < -87, 2.7e-37, 1.2e-38)
        return a, d, 1.01 * ea + cut, 1.01 * ed + cut
    if name == "GELU":
        h, phi = torch.special.erfc(z.abs() / math.sqrt(2)) / 2, torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        a = torch.where(z > 0, z - z * h, z * h)
        d = torch.where(z > 0, 1 - h, h) + z * phi
        r_h = torch.where(z.abs() <= 4, 8e-7, torch.where(z.abs() <= 6, 2e-6, 9e-6))
        far = torch.where(z.abs() > 12.85, 3e-37, 1.2e-38)
        ea = z.abs() * h * r_h + E * a.abs()
        ed = z.abs() * phi * (6 + 1.1 * z * z) * E + h * r_h + torch.where(z > 0, E, 0.0) + E * d.abs()
        # (far out z^2 leaves 64 bits' exponents: phi is 0 and so is its part)
        ed = torch.where(z.abs() > 40, 2 * E * d.abs(), ed)
        return a, d, 1.01 * ea + far, 1.01 * ed + far
    on = (z > 0).double()
    return z * on, on, torch.zeros_like(z), torch.zeros_like(z)


def every_gate(dt):
    """All finite 16-bit values, 64 x 1024, less than 2^100 (fp32 products stay in range)."""
    z = torch.arange(-32768, 32768, device="cuda", dtype=torch.int32).to(torch.int16).view(dt).view(64, 1024).clone()
    z[~(z.double().abs() < 2.0 ** 100)] = 0
    return z


def within(got, ref, bound, z, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    at = int((err - bound).argmax())
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} off, worst at z = {float(z.view(-1)[at]):.6g}: {float(got.reshape(-1)[at]):.9g} for "
                                 f"{float(ref.reshape(-1)[at]):.9g}, bound {float(bound.reshape(-1)[at]):.3g}")


@pytest.mark.parametrize("name", ["SILU", "GELU", "RELU"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("kernel", [None, "tile"])
def test_derivatives_of_every_gate(kernel, dt, name, monkeypatch):
    if kernel:
        monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", kernel)
    g = every_gate(DT[dt])
    T, N = g.shape
    Z = torch.cat([g, torch.ones_like(g)], 1).contiguous()
    dY = torch.zeros((T, 8), device="cuda", dtype=DT[dt])
    W2 = torch.zeros((8, N), device="cuda", dtype=DT[dt])
    dY[:, 0], W2[0] = 1, 1
    with GatedPlan(T, N, 8, DT[dt], "DGATED", act=name, out_f32=True) as p:
        dZ = p.backward(dY, W2, Z)
    z = g.double()
    a, d, ea, ed = bounds(z, name)
    within(dZ[:, :N], d, ed, z, "act'")
    within(dZ[:, N:], a, ea, z, "act")


@pytest.mark.parametrize("name", ["SILU", "GELU", "RELU"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,kernel", [(64, None), (32, None), (16, "warp"), (16, "skinny")])
def test_values_of_every_gate(T, kernel, dt, name, monkeypatch):
    if kernel:
        monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", kernel)
    gates = every_gate(DT[dt])
    X = torch.eye(T, device="cuda", dtype=DT[dt])
    for g in gates.split(T):
        N = g.shape[1]
        W = torch.cat([g, torch.ones_like(g)], 1).contiguous()
        with GatedPlan(T, N, T, DT[dt], "GATED", act=name, out_f32=True) as p:
            H, _ = p.forward(X, W)
        z = g.double()
        a, _, ea, _ = bounds(z, name)
        within(H, a, ea, z, "act")
