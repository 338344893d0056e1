"""Gated layers on the GPU against their definition in 64 bits.

X holds integers in [-3, 3], W integers in [-4, 4] times 2^-4: every product and
fp32 partial sum of Z and dH is exact (multiples of 2^-4 below 2^20), so what is
left are the epilogue's own errors, in units of e = 2^-24:

* RELU: H = max(G, 0) U is one fp32 product: e |H|, then the output's rounding
  (u |H|, u half a step: 2^-8, 2^-11, or e for fp32 outputs).
* SILU: p = 1 / (1 + e^-z). __expf errs by 2 + 1.173 |z| ulp (of 2^-23 relative at
  most), the sum by half an ulp, the reciprocal by 1 ulp, the two products by half an
  ulp each: (12 + 2.4 |z|) e of the result. Below z = -88.72 e^-z exceeds fp32 and p is 0:
  the result misses |z| e^z <= 88.72 x 2^-128 = 2.61e-37 (2 ea counts it: 1.4e-37 each).
* GELU: |z| 2e-7 (the tail's stated 9.3e-8 |z| and the multiply-add), times |U|.
* derivatives: SILU p + a (1 - p): at most (12 + 2.4 |z|) e (1 + 2 |a|) + 4 e (1 + |a|);
  GELU Phi + z phi: h's error 1e-6, phi's exponent z^2 / 2 e: (1e-6 + 4 e) + |z| phi (4 + z^2) e.
  With each the three products of dG: 3 e |dG|.
* dbias: the sum of the elements' bounds, and T e sum |dZ| for the additions.
"""
import math

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GatedPlan, GemmEpiError, Plan, binding

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
E = 2.0 ** -24
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}  # below the normal numbers
ACTS = ["SILU", "GELU", "RELU"]
# T, N, K: one row, ragged rows, features and contraction; several tiles and a part of one
SHAPES = [(1, 8, 8), (3, 72, 24), (17, 200, 136), (100, 264, 520), (128, 64, 192), (129, 136, 72), (300, 520, 264), (700, 1032, 200)]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(shape, hi, g, dt, unit=1.0):
    return (torch.randint(-hi, hi + 1, shape, generator=g, device="cuda") * unit).to(dt)


def guarded(shape, dtype):
    n = math.prod(shape)
    buf = torch.full((n + 512,), 77, dtype=dtype, device="cuda")
    return buf, buf[256:256 + n].view(shape)


def guards_ok(buf):
    return bool((buf[:256] == 77).all()) and bool((buf[-256:] == 77).all())


def act(z, name):
    """act(z), its derivative, and the bounds of the fp32 errors of both."""
    if name == "SILU":
        p = torch.special.expit(z)
        a = z * p
        rel = (12 + 2.4 * z.abs()) * E
        return a, p + a * (1 - p), rel * a.abs() + 1.4e-37, rel * (1 + 2 * a.abs()) + 4 * E * (1 + a.abs())
    if name == "GELU":
        p, phi = torch.special.ndtr(z), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * p, p + z * phi, 2e-7 * z.abs(), 1e-6 + 4 * E + z.abs() * phi * (4 + z * z) * E
    on = (z > 0).double()
    return z * on, on, torch.zeros_like(z), torch.zeros_like(z)


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - bound).max()):.3g} over its bound"


def check_forward(X, W, bias, H, Z, name, w_nk):
    N = H.shape[1]
    z = X.double() @ (W.double().t() if w_nk else W.double())
    if bias is not None:
        z = z + bias.double()
    a, _, ea, _ = act(z[:, :N], name)
    h = a * z[:, N:]
    within(H, h, (U[H.dtype] + 2 * E) * h.abs() + 2 * ea * z[:, N:].abs() + TINY[H.dtype], "H")
    if Z is not None:
        assert torch.equal(Z, z.to(Z.dtype))  # exact, then rounded once


def check_backward(dY, W2, Z, dZ, dbias, name, w_nk):
    N = Z.shape[1] // 2
    dh = dY.double() @ (W2.double().t() if w_nk else W2.double())
    g, up = Z[:, :N].double(), Z[:, N:].double()
    a, d, ea, ed = act(g, name)
    ref = torch.cat([dh * up * d, dh * a], 1)
    own = torch.cat([(dh * up).abs() * ed * 2 + 3 * E * (dh * up * d).abs(), dh.abs() * ea * 2 + 2 * E * (dh * a).abs()], 1)
    within(dZ, ref, (1 + U[dZ.dtype]) * own + U[dZ.dtype] * ref.abs() + TINY[dZ.dtype], "dZ")
    if dbias is not None:
        within(dbias, ref.sum(0), own.sum(0) + (ref.shape[0] + 8) * E * ref.abs().sum(0) + 1e-37, "dbias")


def make(T, N, K, dt, seed, w_nk, bias):
    g = gen(seed)
    X = ints((T, K), 3, g, dt)
    W = ints((2 * N, K) if w_nk else (K, 2 * N), 4, g, dt, 2.0 ** -4)
    b = None if bias is None else ints((2 * N,), 8, g, dt if bias == "16" else torch.float32, 2.0 ** -3)
    return X, W, b


VARIANTS = {"chosen": {}, "tile128": {"KERNEL": "tile", "BN": "128"}, "tile256": {"KERNEL": "tile", "BN": "256"},
            "tile64": {"KERNEL": "tile", "BN": "64"}, "pair": {"KERNEL": "pair"}, "pair whole": {"KERNEL": "pair", "TAIL_SPLIT": "0"}}


def force(monkeypatch, variant):
    for k, v in VARIANTS[variant].items():
        monkeypatch.setenv("GEMM_EPI_" + ("" if k == "TAIL_SPLIT" else "FORCE_") + k, v)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("variant", ["chosen", "tile128", "tile256", "pair", "pair whole"])
def test_forward(shape, variant, monkeypatch):
    T, N, K = shape
    if variant.startswith("pair") and T <= 128:
        pytest.skip("pairs start at 129 rows")
    force(monkeypatch, variant)
    for i, (name, dt, w_nk, bias, aux, f32) in enumerate(
            [("SILU", "bf16", False, None, False, False), ("SILU", "fp16", True, "32", True, False),
             ("GELU", "bf16", True, "16", True, True), ("GELU", "fp16", False, None, True, False),
             ("RELU", "bf16", False, "32", True, True), ("RELU", "fp16", True, "16", False, False)]):
        X, W, b = make(T, N, K, DT[dt], 10 + i, w_nk, bias)
        hb, H = guarded((T, N), torch.float32 if f32 else DT[dt])
        zb, Z = guarded((T, 2 * N), DT[dt])
        with GatedPlan(T, N, K, DT[dt], "GATED_AUX" if aux else "GATED", act=name, w_nk=w_nk, out_f32=f32) as p:
            if bias == "32":
                p.set_bias_f32()
            kernel = p.info()["kernel"]
            assert kernel == {"chosen": kernel, "pair": 2, "pair whole": 2}.get(variant, 0) and (variant != "chosen" or (kernel == 1) == (T <= 32))
            p.gemm_epi_gated_execute(X, W, b, H, Z)
            first = H.clone()
            p.gemm_epi_gated_execute(X, W, b, H, Z)
            torch.cuda.synchronize()
            assert p.status() == 0
        assert torch.equal(first, H) and guards_ok(hb) and guards_ok(zb)
        assert aux or bool((Z == 77).all())
        check_forward(X, W, b, H, Z if aux else None, name, w_nk)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("variant", ["chosen", "tile64", "tile128", "tile256", "pair", "pair whole"])
def test_backward(shape, variant, monkeypatch):
    T, N, K = shape
    if variant.startswith("pair") and T <= 128:
        pytest.skip("pairs start at 129 rows")
    force(monkeypatch, variant)
    for i, (name, dt, w_nk, with_b, f32) in enumerate(
            [("SILU", "bf16", False, True, False), ("SILU", "fp16", True, False, True), ("GELU", "bf16", True, True, True),
             ("GELU", "fp16", False, True, False), ("RELU", "bf16", True, False, False), ("RELU", "fp16", False, True, True)]):
        g = gen(40 + i)
        dY = ints((T, K), 3, g, DT[dt])
        W2 = ints((N, K) if w_nk else (K, N), 4, g, DT[dt], 2.0 ** -4)
        Z = (2 * torch.randn((T, 2 * N), generator=g, device="cuda")).to(DT[dt])
        Z[:, ::7] = 0  # where RELU's derivative jumps
        db, dZ = guarded((T, 2 * N), torch.float32 if f32 else DT[dt])
        bb, dbias = guarded((2 * N,), torch.float32)
        with GatedPlan(T, N, K, DT[dt], "DGATED", act=name, w_nk=w_nk, out_f32=f32) as p:
            kernel = p.info()["kernel"]
            assert kernel == {"chosen": kernel, "pair": 2, "pair whole": 2}.get(variant, 0)
            p.gemm_epi_dgated_execute(dY, W2, Z, dZ, dbias if with_b else None)
            first, first_b = dZ.clone(), dbias.clone()
            p.gemm_epi_dgated_execute(dY, W2, Z, dZ, dbias if with_b else None)
            torch.cuda.synchronize()
            assert p.status() == 0
        assert torch.equal(first, dZ) and torch.equal(first_b, dbias) and guards_ok(db) and guards_ok(bb)
        assert with_b or bool((dbias == 77).all())
        check_backward(dY, W2, Z, dZ, dbias if with_b else None, name, w_nk)


@pytest.mark.parametrize("T,N,K", [(1, 8, 8), (2, 24, 40), (7, 72, 104), (8, 2048, 1024), (9, 40, 32), (13, 2376, 264), (16, 1032, 520),
                                   (3, 4752, 96), (5, 7112, 64), (16, 16 * 16 * 148 + 8, 40), (1, 16, 16384), (16, 48, 10008)])
@pytest.mark.parametrize("kernel", ["warp", "skinny"])
def test_few_rows_on_either_kernel(T, N, K, kernel, monkeypatch):
    """Half rows of tiles, one to more than sixteen a CTA; contractions that clusters share."""
    monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", kernel)
    for i, (name, dt, w_nk, bias, aux, f32) in enumerate(
            [("SILU", "bf16", False, None, False, False), ("GELU", "fp16", True, "32", True, False),
             ("RELU", "bf16", True, "16", True, True), ("SILU", "fp16", False, "16", True, True)]):
        X, W, b = make(T, N, K, DT[dt], 20 + i, w_nk, bias)
        hb, H = guarded((T, N), torch.float32 if f32 else DT[dt])
        zb, Z = guarded((T, 2 * N), DT[dt])
        with GatedPlan(T, N, K, DT[dt], "GATED_AUX" if aux else "GATED", act=name, w_nk=w_nk, out_f32=f32) as p:
            if bias == "32":
                p.set_bias_f32()
            assert p.info()["kernel"] == 1 and (p.info()["tile_m"] == 32) == (kernel == "warp")
            assert K < 16384 or p.info()["split_k"] > 1
            p.gemm_epi_gated_execute(X, W, b, H, Z)
            first = H.clone()
            p.gemm_epi_gated_execute(X, W, b, H, Z)
            torch.cuda.synchronize()
            assert p.status() == 0
        assert torch.equal(first, H) and guards_ok(hb) and guards_ok(zb)
        assert aux or bool((Z == 77).all())
        check_forward(X, W, b, H, Z if aux else None, name, w_nk)


@pytest.mark.parametrize("T,N,K,grid", [(8, 64, 2048, "7"), (31, 136, 1032, "11"), (17, 72, 520, "3"), (32, 200, 4096, "61"),
                                        (5, 9600, 264, "70"), (32, 9800, 520, "140"), (16, 19200, 264, "33")])
@pytest.mark.parametrize("w_nk", [False, True])
def test_few_rows_shared_tiles(T, N, K, grid, w_nk, monkeypatch):
    """Tiles shared by up to many CTAs: their parts are summed in a fixed order."""
    monkeypatch.setenv("GEMM_EPI_SKINNY_GRID", grid)
    X, W, b = make(T, N, K, torch.bfloat16, 3, w_nk, "16")
    with GatedPlan(T, N, K, torch.bfloat16, "GATED_AUX", act="SILU", w_nk=w_nk) as p:
        assert p.info()["kernel"] == 1 and p.info()["split_k"] > 1
        H, Z = p.forward(X, W, b)
        for _ in range(5):
            H2, Z2 = p.forward(X, W, b)
            assert torch.equal(H, H2) and torch.equal(Z, Z2)
        assert p.status() == 0
    check_forward(X, W, b, H, Z, "SILU", w_nk)


@pytest.mark.parametrize("name", ACTS)
def test_values_over_the_whole_range(name):
    """G is given (X = I): values to +-60, tiny ones, zeros, infinities and NaN; U = 1 and 3."""
    T = K = 64
    N = 512
    v = torch.cat([torch.linspace(-60, 60, T * N // 2, device="cuda"),
                   10.0 ** torch.linspace(-7, 1, T * N // 4, device="cuda"), -10.0 ** torch.linspace(-7, 1, T * N // 4, device="cuda")])
    g = v.view(K, N).to(torch.bfloat16)
    W = torch.cat([g, torch.full((K, N), 3.0, device="cuda", dtype=torch.bfloat16)], 1).contiguous()
    X = torch.eye(T, device="cuda", dtype=torch.bfloat16)
    X[5] = 0  # a row of zeros
    with GatedPlan(T, N, K, torch.bfloat16, "GATED_AUX", act=name, out_f32=True) as p:
        H, Z = p.forward(X, W)
    check_forward(X, W, None, H, Z, name, False)
    # special values: the rows' own G, with no contraction across them (dY2 = I)
    dY = torch.eye(T, device="cuda", dtype=torch.bfloat16)
    W2 = torch.ones((K, N), device="cuda", dtype=torch.bfloat16)
    with GatedPlan(T, N, K, torch.bfloat16, "DGATED", act=name, out_f32=True) as p:
        dZ, dbias = p.backward(dY, W2, Z, with_dbias=True)
        check_backward(dY, W2, Z, dZ, dbias, name, False)
        odd = Z.clone()
        odd[1, 0], odd[1, 1], odd[1, 2] = float("inf"), float("nan"), -200.0
        odd[2, N], odd[2, N + 1] = float("inf"), float("nan")
        got = p.backward(dY, W2, odd)
    same = torch.ones_like(dZ, dtype=torch.bool)
    for r, c in ((1, 0), (1, 1), (1, 2), (2, 0), (2, 1)):
        same[r, c] = same[r, N + c] = False
    assert torch.equal(got[same], dZ[same])  # nothing spreads
    assert got[1, N] == float("inf") and bool(got[1, N + 1].isnan()) == (name != "RELU")
    # (act(-200) = 0; U's infinity reaches dG alone)
    assert abs(float(got[1, 2])) < 1e-30 and abs(float(got[1, N + 2])) < 1e-30
    assert torch.equal(got[2, N:N + 2], dZ[2, N:N + 2])


def test_rows_beyond_32_bit_offsets():
    T, N, K = 140000, 8200, 64
    g = gen(9)
    X, W = ints((T, K), 3, g, torch.bfloat16), ints((K, 2 * N), 4, g, torch.bfloat16, 2.0 ** -4)
    with GatedPlan(T, N, K, torch.bfloat16, "GATED_AUX") as p:
        H, Z = p.forward(X, W)
    rows = torch.tensor([0, 1, 70001, 131071, 131072, 139998, 139999], device="cuda")
    check_forward(X[rows], W, None, H[rows], Z[rows], "SILU", False)
    dY, W2 = ints((T, K), 3, g, torch.bfloat16), ints((K, N), 4, g, torch.bfloat16, 2.0 ** -4)
    del H
    with GatedPlan(T, N, K, torch.bfloat16, "DGATED") as p:
        dZ = p.backward(dY, W2, Z)
    check_backward(dY[rows], W2, Z[rows], dZ[rows], None, "SILU", False)


def test_not_finite_weights_stay_in_their_features():
    """Rows past T of the last tile are zeros times the weight: an infinite one must not reach the sums."""
    T, N, K = 70, 72, 64
    g = gen(2)
    dY, W2 = torch.ones((T, K), device="cuda", dtype=torch.bfloat16), ints((K, N), 4, g, torch.bfloat16, 2.0 ** -4)
    Z = torch.ones((T, 2 * N), device="cuda", dtype=torch.bfloat16)
    W2[3, 5] = float("inf")
    with GatedPlan(T, N, K, torch.bfloat16, "DGATED", act="RELU") as p:
        dZ, dbias = p.backward(dY, W2, Z, with_dbias=True)
    on = torch.arange(2 * N, device="cuda") % N == 5
    assert bool((dbias[on] == float("inf")).all()) and bool((dZ[:, on] == float("inf")).all())
    assert bool(dbias[~on].isfinite().all())


@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("name", ACTS)
def test_block_step_against_autograd(T, name):
    """A whole block, [out, in] weights: H of the gated layer, Y = H Wd^T; dZ and the biases' gradient by
    DGATED, dX by NONE over 2N, dW by WGRAD. Operands are rounded to bf16 where the library stores
    them: Z, H and dZ (each relative 2^-8; dZ sees Z's rounding through act'), so 3 x 2^-8 of the sums of magnitudes."""
    N, K = 136, 200
    bf = torch.bfloat16
    X, W, b = make(T, N, K, bf, 21, True, "16")
    Wd = ints((K, N), 4, gen(22), bf, 2.0 ** -4)
    dY = ints((T, K), 3, gen(23), bf)
    with GatedPlan(T, N, K, bf, "GATED_AUX", act=name, w_nk=True) as f, GatedPlan(T, N, K, bf, "DGATED", act=name) as d, \
            Plan(T, K, 2 * N, bf, "NONE", out_f32=True) as dx, Plan(T, K, 2 * N, bf, "WGRAD", out_f32=True) as dw, \
            Plan(T, K, N, bf, "NONE", w_nk=True, out_f32=True) as down:
        H, Z = f.forward(X, W, b)
        Y, _ = down.forward(H, Wd, None)
        dZ, dbias = d.backward(dY, Wd, Z, with_dbias=True)
        dX, _ = dx.forward(dZ, W, None)
        dW = dw.wgrad(dZ, X)  # 2N x K
        torch.cuda.synchronize()
    x, w, bb, wd = (t.double().requires_grad_() for t in (X, W, b, Wd))
    z = x @ w.t() + bb
    a = {"SILU": torch.nn.functional.silu, "GELU": torch.nn.functional.gelu, "RELU": torch.relu}[name](z[:, :N])
    y = (a * z[:, N:]) @ wd.t()
    y.backward(dY.double())
    tol = 3 * 2.0 ** -8
    dh = (dY.double() @ wd.detach()).abs()
    zmag = z.detach().abs()
    # |act'| <= 1.13, |act''| <= 1: what one rounding of G and of U moves dZ by
    move = torch.cat([dh * (1.13 * zmag[:, N:] + zmag[:, N:] * zmag[:, :N]), 1.13 * dh * zmag[:, :N]], 1) * tol
    within(Y, y.detach(), tol * ((a * z[:, N:]).detach().abs() @ wd.detach().abs().t()) + 1e-6, "Y")
    within(dX, x.grad, move @ w.detach().abs() + 1e-6, "dX")
    within(dW, w.grad, move.t() @ x.detach().abs() + 1e-6, "dW")
    within(dbias, bb.grad, move.sum(0) + 1e-6, "dbias")


@pytest.mark.parametrize("name", ["SILU", "GELU"])
def test_backward_against_differences(name):
    """dZ of one element at a time against central differences of H in 64 bits (truncation h^2 / 6 |act'''|
    with |act'''| < 1.2 and h = 1e-3, below 1e-6 |dH U|)."""
    T, N, K = 40, 64, 32
    dY, W2 = ints((T, K), 3, gen(1), torch.bfloat16), ints((K, N), 4, gen(2), torch.bfloat16, 2.0 ** -4)
    Z = torch.randn((T, 2 * N), generator=gen(3), device="cuda").to(torch.bfloat16)
    with GatedPlan(T, N, K, torch.bfloat16, "DGATED", act=name, out_f32=True) as p:
        dZ = p.backward(dY, W2, Z)
    dh, g, up, h = dY.double() @ W2.double(), Z[:, :N].double(), Z[:, N:].double(), 1e-3
    num_g = dh * up * (act(g + h, name)[0] - act(g - h, name)[0]) / (2 * h)
    num_u = dh * act(g, name)[0] * ((up + h) - (up - h)) / (2 * h)
    within(dZ[:, :N], num_g, 4e-6 * (dh * up).abs() + 1e-9, "dG")
    within(dZ[:, N:], num_u, 4e-6 * dh.abs() * (1 + g.abs()) + 1e-9, "dU")


@pytest.mark.parametrize("T,N,K", [(4, 200, 256), (300, 520, 264)])
def test_streams_and_graphs(T, N, K):
    X, W, b = make(T, N, K, torch.bfloat16, 5, False, "16")
    W2, dY = ints((K, N), 4, gen(6), torch.bfloat16, 2.0 ** -4), ints((T, K), 3, gen(7), torch.bfloat16)
    f, d = GatedPlan(T, N, K, torch.bfloat16, "GATED_AUX"), GatedPlan(T, N, K, torch.bfloat16, "DGATED")
    H, Z = f.forward(X, W, b)
    dZ, db = d.backward(dY, W2, Z, with_dbias=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    H1, Z1 = f.forward(X, W, b, stream=s)
    dZ1, db1 = d.backward(dY, W2, Z1, with_dbias=True, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in ((H, H1), (Z, Z1), (dZ, dZ1), (db, db1)))
    outs = [torch.zeros_like(t) for t in (H, Z, dZ, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.gemm_epi_gated_execute(X, W, b, outs[0], outs[1])
        d.gemm_epi_dgated_execute(dY, W2, outs[1], outs[2], outs[3])
    for seed in (30, 31):
        X.copy_(ints((T, K), 3, gen(seed), torch.bfloat16))
        graph.replay()
        H, Z = f.forward(X, W, b)
        dZ, db = d.backward(dY, W2, Z, with_dbias=True)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, (H, Z, dZ, db)))
    assert f.status() == 0 and d.status() == 0


@pytest.mark.parametrize("kernel,T", [("skinny", 20), ("tile", 300), ("pair", 300)])
def test_watchdog_reports_and_the_plan_recovers(kernel, T, monkeypatch):
    """A withheld completion signal runs a bounded wait out; a new plan is not disturbed."""
    N, K = 264, 512
    X, W, b = make(T, N, K, torch.bfloat16, 5, False, None)
    if kernel != "skinny":
        monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", kernel)
    monkeypatch.setenv("GEMM_EPI_WAIT_TIMEOUT_MS", "50")
    monkeypatch.setenv("GEMM_EPI_TEST_HOOKS", "1")
    monkeypatch.setenv("GEMM_EPI_INJECT_STALL", "1")
    with GatedPlan(T, N, K, torch.bfloat16) as p:
        p.forward(X, W)
        torch.cuda.synchronize()
        assert p.status() == binding.ERR_TIMEOUT and p.status() == 0
    if kernel != "skinny":
        with GatedPlan(T, N, K, torch.bfloat16, "DGATED") as p:
            p.backward(X, torch.zeros((K, N), device="cuda", dtype=torch.bfloat16),
                       torch.zeros((T, 2 * N), device="cuda", dtype=torch.bfloat16), with_dbias=True)
            torch.cuda.synchronize()
            assert p.status() == binding.ERR_TIMEOUT
    monkeypatch.delenv("GEMM_EPI_INJECT_STALL")
    with GatedPlan(T, N, K, torch.bfloat16) as p:
        H, _ = p.forward(X, W)
        torch.cuda.synchronize()
        assert p.status() == 0
    check_forward(X, W, None, H, None, "SILU", False)


def test_refusals():
    bf = torch.bfloat16
    X, W = torch.zeros((4, 64), device="cuda", dtype=bf), torch.zeros((64, 128), device="cuda", dtype=bf)
    H, Z = torch.zeros((4, 64), device="cuda", dtype=bf), torch.zeros((4, 128), device="cuda", dtype=bf)
    with GatedPlan(4, 64, 64, bf, "GATED_AUX") as f, GatedPlan(4, 64, 64, bf, "DGATED") as d, Plan(4, 64, 64, bf, "NONE") as q:
        with pytest.raises(GemmEpiError) as e:
            f.gemm_epi_gated_execute(X, W, None, H)  # no aux
        assert e.value.code == binding.ERR_EPILOG_MISMATCH
        L = binding.lib()
        ptr = [t.data_ptr() for t in (X, W, H, Z)]
        assert L.gemm_epi_gated_execute(d.handle, ptr[0], ptr[1], None, ptr[2], None, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_dgated_execute(f.handle, ptr[0], ptr[1], ptr[3], ptr[3], None, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_gated_execute(q.handle, ptr[0], ptr[1], None, ptr[2], None, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_execute(f.handle, ptr[0], ptr[1], None, ptr[2], None, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_gated_execute(f.handle, ptr[0] + 2, ptr[1], None, ptr[2], ptr[3], None) == binding.ERR_MISALIGNED
        assert L.gemm_epi_gated_execute(f.handle, ptr[0], ptr[1], ptr[0] + 1, ptr[2], ptr[3], None) == binding.ERR_MISALIGNED
        assert L.gemm_epi_gated_execute(f.handle, None, ptr[1], None, ptr[2], ptr[3], None) == binding.ERR_INVALID_ARG
        assert L.gemm_epi_dgated_execute(d.handle, ptr[0], ptr[1], None, ptr[3], None, None) == binding.ERR_INVALID_ARG
        assert L.gemm_epi_set_bias_f32(d.handle, 1) == binding.ERR_EPILOG_MISMATCH
        for bad in (W.t(), W[:, :64], W.float(), W.cpu()):
            with pytest.raises(ValueError):
                f.gemm_epi_gated_execute(X, bad, None, H, Z)
