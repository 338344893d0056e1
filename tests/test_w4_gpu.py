"""4-bit weights with group scales on the GPU: codes, layout and products against
their definition in 64 bits.

Exact products: X holds integers in [-3, 3] and the scales are powers of two in a
narrow range, so that every product, group sum and feature sum is exact in fp32 (multiples
of 2^-6 below 2^18) and Y has one right value, rounded once.

Products of other scales: a group's sum of up to 128 exact products errs by at most
128 x 2 e of its magnitudes (e = 2^-24; 2 for a truncating adder), the groups' sums,
scaled and added, by (K / G + 8) e more: (2 x 128 + K / G + 8) e S, S the sum of |x w|;
then the epilog's own errors (its bounds as derived for gated layers) and one rounding
of u |Y|.
"""
import math

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import (GemmEpiError, Plan, W4Plan, binding, gemm_epi_w4_dequantize, gemm_epi_w4_pack,
                                         gemm_epi_w4_quantize, w4_empty, w4_pack, w4_quantize)

from test_gated_gpu import E, TINY, U, act, gen, guarded, guards_ok, ints, within

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def reference_codes(W, G, zeros):
    """Codes, scales (rounded), zeros of W [N, K] in 64 bits."""
    w = W.double().view(W.shape[0], -1, G)
    lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15 if zeros else w.abs().amax(-1) / 7).float().to(W.dtype)
    d = torch.where(s > 0, s, 1).double()[..., None]
    z = (-lo[..., None] / d).round().clamp(0, 15) if zeros else torch.full_like(d, 8.0)
    z = torch.where(s[..., None] > 0, z, 0.0 if zeros else 8.0)
    c = ((w / d).round() + z).clamp(0, 15)
    c = torch.where(s[..., None] > 0, c, z.expand_as(c))
    return c.view(W.shape).to(torch.uint8), s, z[..., 0].to(torch.uint8)


def unpack(q, s, z, N, K, G):
    """The layout, as the header states it -> row-major codes, scales, zeros."""
    kt, ng = (K + 127) // 128, 128 // G
    n = torch.arange(N, device="cuda")[:, None]
    k = torch.arange(K, device="cuda")[None, :]
    tile, f, c = (n // 32) * kt + k // 128, n % 32, k % 128
    word = 2048 * tile + 512 * (c // 32) + 16 * f + 4 * (c % 32 // 8)
    bit = 4 * (c % 8 // 2) + 16 * (c % 2)
    codes = (q.long()[word + bit // 8] >> (bit % 8)) & 15
    k = torch.arange(K // G, device="cuda")[None, :]
    at = 32 * (ng * ((n // 32) * kt + k // ng) + k % ng) + f
    return codes.to(torch.uint8), s[at], None if z is None else z[at]


def rowmajor(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()


def weights(N, K, G, dt, seed, zeros, exact, batch=None):
    """Codes, scales, zeros as a checkpoint has them."""
    g = gen(seed)
    shape = (N,) if batch is None else (batch, N)
    codes = torch.randint(0, 16, (*shape, K), generator=g, device="cuda", dtype=torch.uint8)
    if exact:
        s = 2.0 ** torch.randint(-6, -3, (*shape, K // G), generator=g, device="cuda")
    else:
        s = (torch.rand((*shape, K // G), generator=g, device="cuda") + 0.5) / (5 * math.sqrt(K))
    z = torch.randint(0, 16, (*shape, K // G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, s.to(dt), z


def values(codes, s, z, G):
    q = codes.double().view(*s.shape, G) - (8.0 if z is None else z.double()[..., None])
    return (q * s.double()[..., None]).view(codes.shape)


@pytest.mark.parametrize("N,K,G", [(1, 32, 32), (16, 128, 128), (17, 160, 32), (40, 192, 64), (200, 1024, 128), (1000, 352, 32)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_quantize_matches_the_definition(N, K, G, zeros, dt):
    dt = DT[dt]
    W = (torch.randn((N, K), generator=gen(N + K), device="cuda") / 8).to(dt)
    W.view(-1)[torch.randperm(N * K, generator=gen(1), device="cuda")[:N * K // 50]] *= 8
    if N > 2:
        W[0] = 0                                    # groups of zeros
        W[1] = W[1].abs()                           # one sign alone
        W[2] = torch.finfo(dt).tiny * 3             # scales below the normal numbers
    q, s, z = w4_empty(N, K, dt, G, zeros)
    guards = [torch.full((t.numel() + 128,), 99 if t.dtype == torch.uint8 else 99.0, dtype=t.dtype, device="cuda") for t in (q, s)]
    q, s = guards[0][64:64 + q.numel()], guards[1][64:64 + s.numel()]
    gemm_epi_w4_quantize(W, q, s, z, group=G)
    for b, t in zip(guards, (q, s)):
        assert bool((b[:64] == 99).all()) and bool((b[64 + t.numel():] == 99).all())
    codes, sc, ze = unpack(q, s, z, N, K, G)
    rc, rs, rz = reference_codes(W, G, zeros)
    assert torch.equal(sc, rs) and torch.equal(codes, rc) and (z is None or torch.equal(ze, rz))
    out = torch.empty((N, K), dtype=torch.float32, device="cuda")
    gemm_epi_w4_dequantize(q, s, z, out, group=G)
    ref = values(rc, rs, rz if zeros else None, G)
    assert torch.equal(out.double(), ref)
    out16 = torch.empty((N, K), dtype=dt, device="cuda")
    gemm_epi_w4_dequantize(q, s, z, out16, group=G)
    assert torch.equal(out16, ref.float().to(dt))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_quantize_ties_and_every_pattern(dt):
    """Every finite 16-bit value with a maximum of 7 x a scale beside it: quotients that are ties (w = (m + 1/2) s)
    among them; then groups with an infinity or NaN."""
    dt = DT[dt]
    bits = torch.arange(-32768, 32768, device="cuda", dtype=torch.int32).to(torch.int16).view(dt)
    bits = bits[bits.isfinite()]
    for scale in (1.0, 0.75, 2.0 ** -10, 3.0 * 2.0 ** 7):
        v = bits[bits.abs().double() <= 7 * scale]
        v = torch.cat([v, torch.zeros((-len(v)) % 31, dtype=dt, device="cuda")]).view(-1, 31)
        top = torch.full((len(v), 1), 7 * scale, device="cuda").to(dt)
        W = torch.cat([v, top], 1).contiguous()
        q, s, _ = w4_quantize(W, group=32)
        codes, sc, _ = unpack(q, s, None, *W.shape, 32)
        rc, rs, _ = reference_codes(W, 32, False)
        assert torch.equal(sc, rs) and torch.equal(codes, rc)
    W = torch.ones((4, 64), dtype=dt, device="cuda")
    W[0, 3], W[1, 40], W[2, 5] = float("inf"), float("nan"), float("-inf")
    for zeros in (False, True):
        q, s, z = w4_quantize(W, group=32, zeros=zeros)
        out = torch.empty((4, 64), device="cuda")
        gemm_epi_w4_dequantize(q, s, z, out, group=32)
        nan = torch.zeros((4, 64), dtype=torch.bool, device="cuda")
        nan[0, :32] = nan[1, 32:] = nan[2, :32] = True
        assert torch.equal(out.isnan(), nan)


@pytest.mark.parametrize("N,K,G,batch", [(1, 32, 32, None), (24, 96, 32, 3), (100, 320, 64, 2), (33, 1152, 128, None)])
@pytest.mark.parametrize("zeros", [False, True])
def test_pack_is_the_layout(N, K, G, batch, zeros):
    codes, s, z = weights(N, K, G, torch.float16, 5, zeros, False, batch)
    q, ps, pz = w4_pack(rowmajor(codes), s, z)
    out = torch.empty(codes.shape, dtype=torch.float32, device="cuda")
    gemm_epi_w4_dequantize(q, ps, pz, out, group=G)
    assert torch.equal(out.double(), values(codes, s, z, G))
    if batch is None:
        uc, us, uz = unpack(q, ps, pz, N, K, G)
        assert torch.equal(uc, codes) and torch.equal(us, s) and (z is None or torch.equal(uz, z))


# T around the tiles' 8, 16, 32, 64 rows and over; ragged N and K, a K of several slices
CASES = [(1, 8, 32, 32), (1, 200, 1024, 128), (3, 72, 160, 32), (8, 520, 2048, 64), (9, 264, 1152, 128), (16, 136, 4160, 32),
         (17, 1000, 512, 128), (32, 72, 4096, 64), (33, 264, 1024, 32), (48, 2056, 2080, 32), (64, 200, 2176, 128), (65, 136, 640, 64),
         (130, 72, 4096, 128), (256, 24, 256, 32)]


@pytest.mark.parametrize("T,N,K,G", CASES)
@pytest.mark.parametrize("zeros", [False, True])
def test_products_exact(T, N, K, G, zeros):
    for dt, epi, f32, bias in (("bf16", "NONE", True, None), ("fp16", "RELU_BIAS", False, "16"), ("bf16", "BIAS", False, "32"),
                               ("fp16", "NONE", False, None)):
        dt = DT[dt]
        codes, s, z = weights(N, K, G, dt, T + N, zeros, True)
        X = ints((T, K), 3, gen(T), dt)
        b = None if bias is None else ints((N,), 8, gen(2), dt if bias == "16" else torch.float32, 2.0 ** -3)
        w4 = w4_pack(rowmajor(codes), s, z)
        yb, Y = guarded((T, N), torch.float32 if f32 else dt)
        with W4Plan(T, N, K, dt, epi, group=G, out_f32=f32) as p:
            if bias == "32":
                p.set_bias_f32()
            assert p.info()["kernel"] == 8 and p.info()["launches"] == 1
            p.gemm_epi_w4_execute(X, *w4, b, Y)
            first = Y.clone()
            p.gemm_epi_w4_execute(X, *w4, b, Y)
            torch.cuda.synchronize()
            assert p.status() == 0
        ref = X.double() @ values(codes, s, z, G).t() + (0 if b is None else b.double())
        if epi == "RELU_BIAS":
            ref = ref.clamp(min=0)
        assert guards_ok(yb) and torch.equal(first, Y)
        assert torch.equal(Y, ref.float().to(Y.dtype))


@pytest.mark.parametrize("T,N,K,G", CASES)
@pytest.mark.parametrize("zeros", [False, True])
def test_products_of_any_scales(T, N, K, G, zeros):
    for dt, epi, name, f32, with_b in (("bf16", "GATED", "SILU", False, False), ("fp16", "GATED", "GELU", True, True),
                                       ("fp16", "GELU_BIAS", "SILU", False, True), ("bf16", "NONE", "SILU", True, False),
                                       ("fp16", "GATED", "RELU", False, True)):
        dt = DT[dt]
        gated = epi == "GATED"
        codes, s, z = weights(N, K, G, dt, T + N, zeros, False, 2 if gated else None)
        X = torch.randn((T, K), generator=gen(T), device="cuda").to(dt)
        b = torch.randn(((2 if gated else 1) * N,), generator=gen(3), device="cuda").to(dt) if with_b else None
        w4 = w4_pack(rowmajor(codes), s, z)
        with W4Plan(T, N, K, dt, epi, group=G, act=name, out_f32=f32) as p:
            Y = p.forward(X, *w4, bias=b)
            assert torch.equal(Y, p.forward(X, *w4, bias=b))
        w = values(codes, s, z, G).reshape(-1, K)
        y, size = X.double() @ w.t(), X.double().abs() @ w.abs().t()
        if b is not None:
            y = y + b.double()
            size = size + b.double().abs()
        err = (2 * 128 + K / G + 8) * E * size
        u = U[Y.dtype]
        if not gated:
            if epi == "GELU_BIAS":
                a, d, ea, _ = act(y, "GELU")
                err, y = 1.13 * err + 2 * ea, a  # |GELU'| <= 1.13
            within(Y, y, (1 + u) * err + u * y.abs() + TINY[Y.dtype], epi)
            continue
        g, up, eg, eu = y[:, :N], y[:, N:], err[:, :N], err[:, N:]
        a, d, ea, _ = act(g, name)
        if name == "RELU":
            ea = ea + 0  # (at 0 either side is within |g|'s own error)
        # |act'| <= 1.13; the products of both errors count with 2
        bound = (1.13 * eg + 2 * ea) * (up.abs() + 2 * eu) + eu * a.abs()
        within(Y, a * up, (1 + u) * bound + (u + 2 * E) * (a * up).abs() + TINY[Y.dtype], "gated " + name)


@pytest.mark.parametrize("T,N,K,G", CASES)
@pytest.mark.parametrize("kernel", ["warp", "tmem"])
def test_products_on_either_kernel(kernel, T, N, K, G, monkeypatch):
    monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", kernel)
    with W4Plan(T, N, K, torch.bfloat16, "NONE", group=G) as p:
        assert p.info()["tile_m"] == {"warp": 32, "tmem": 128}[kernel]
    for zeros in (False, True):
        test_products_exact(T, N, K, G, zeros)
        test_products_of_any_scales(T, N, K, G, zeros)


@pytest.mark.parametrize("N", [8, 16, 24, 2368, 2376, 4752, 4744, 7112, 16 * 16 * 148 + 8])
@pytest.mark.parametrize("T", [1, 9, 37])
def test_shares_of_half_tiles(N, T, monkeypatch):
    """Half rows of tiles, one to sixteen and more a CTA, of one to five columns of tiles."""
    monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", "warp")
    dt = torch.float16
    for K in (32, 384, 640):
        codes, s, z = weights(N, K, 32, dt, N + K, True, True, 2)
        w4 = w4_pack(rowmajor(codes), s, z)
        X = ints((T, K), 3, gen(T), dt)
        y = X.double() @ values(codes, s, z, 32).reshape(-1, K).t()
        with W4Plan(T, N, K, dt, "GATED", group=32, act="RELU", out_f32=True) as p:
            Y = p.forward(X, *w4)
            assert torch.equal(Y, p.forward(X, *w4))
        r = y[:, :N].clamp(min=0) * y[:, N:]
        within(Y, r, 2 * E * r.abs(), "gated")  # one fp32 product of exact sums
        with W4Plan(T, N, K, dt, "NONE", group=32, out_f32=True) as p:
            Y = p.forward(X, *w4_pack(rowmajor(codes[0].contiguous()), s[0].contiguous(), z[0].contiguous()))
        assert torch.equal(Y.double(), y[:, :N])


@pytest.mark.parametrize("kernel", ["warp", "tmem"])
@pytest.mark.parametrize("T,N,K", [(1, 8, 32768), (8, 48, 16384), (13, 80, 16384), (30, 16, 24576)])
def test_columns_shared_by_clusters(T, N, K, kernel, monkeypatch):
    monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", kernel)
    dt = torch.bfloat16
    codes, s, z = weights(N, K, 128, dt, T, True, True, 2)
    w4 = w4_pack(rowmajor(codes), s, z)
    X = ints((T, K), 2, gen(T), dt)
    y = X.double() @ values(codes, s, z, 128).reshape(-1, K).t()
    with W4Plan(T, N, K, dt, "GATED", group=128, act="RELU", out_f32=True) as p:
        assert p.info()["split_k"] > 1
        Y = p.forward(X, *w4)
        assert torch.equal(Y, p.forward(X, *w4))
    r = y[:, :N].clamp(min=0) * y[:, N:]
    within(Y, r, 2 * E * r.abs(), "gated")  # one fp32 product of exact sums
    with W4Plan(T, N, K, dt, "NONE", group=128, out_f32=True) as p:
        Y = p.forward(X, *w4_pack(rowmajor(codes[0].contiguous()), s[0].contiguous(), z[0].contiguous()))
    assert torch.equal(Y.double(), y[:, :N])


def test_wide_weight_and_many_tiles():
    """A vocabulary's worth of features, few columns: many tiles a CTA."""
    T, N, K, G = 2, 50000, 128, 128
    codes, s, z = weights(N, K, G, torch.bfloat16, 1, True, True)
    X = ints((T, K), 3, gen(1), torch.bfloat16)
    with W4Plan(T, N, K, torch.bfloat16, "NONE", group=G, out_f32=True) as p:
        Y = p.forward(X, *w4_pack(rowmajor(codes), s, z))
    assert torch.equal(Y.double(), X.double() @ values(codes, s, z, G).t())


def test_long_contraction():
    """K of 65 536, shared by many CTAs."""
    T, N, K, G = 8, 40, 65536, 64
    codes, s, z = weights(N, K, G, torch.float16, 1, False, True)
    X = ints((T, K), 2, gen(1), torch.float16)
    with W4Plan(T, N, K, torch.float16, "NONE", group=G, out_f32=True) as p:
        assert p.info()["split_k"] > 1
        Y = p.forward(X, *w4_pack(rowmajor(codes), s, z))
    assert torch.equal(Y.double(), X.double() @ values(codes, s, z, G).t())


def test_rows_do_not_mix():
    """A row of NaN and infinities stays in its row of Y; zero points of 127 and 0."""
    T, N, K, G = 12, 72, 256, 32
    codes, s, _ = weights(N, K, G, torch.bfloat16, 1, False, True)
    z = torch.full((N, K // G), 127, dtype=torch.uint8, device="cuda")
    z[::2] = 0
    X = ints((T, K), 3, gen(1), torch.bfloat16)
    bad = X.clone()
    bad[3, 5], bad[7] = float("nan"), float("inf")
    w4 = w4_pack(rowmajor(codes), s, z)
    with W4Plan(T, N, K, torch.bfloat16, "NONE", group=G, out_f32=True) as p:
        Y, Yb = p.forward(X, *w4), p.forward(bad, *w4)
    assert torch.equal(Y.double(), X.double() @ values(codes, s, z, G).t())
    assert bool(Yb[3].isnan().all())
    keep = [t for t in range(T) if t not in (3, 7)]
    assert torch.equal(Yb[keep], Y[keep])


def test_prompt_through_the_same_weight():
    """More rows than the plan takes: dequantised to 16 bits, a dense plan with an N x K weight; few rows of the
    same prompt through the 4-bit plan agree with it (the weight's rounding: u per product, then one rounding each)."""
    T, N, K, G = 300, 264, 512, 64
    dt = torch.bfloat16
    W = (torch.randn((N, K), generator=gen(1), device="cuda") / 16).to(dt)
    q, s, z = w4_quantize(W, group=G, zeros=True)
    held = torch.empty_like(W)
    gemm_epi_w4_dequantize(q, s, z, held, group=G)
    X = torch.randn((T, K), generator=gen(2), device="cuda").to(dt)
    with pytest.raises(GemmEpiError, match="dequantize"):
        W4Plan(T, N, K, dt, "NONE", group=G)
    with Plan(T, N, K, dt, "NONE", w_nk=True) as d, W4Plan(5, N, K, dt, "NONE", group=G) as p:
        Y, _ = d.forward(X, held, None)
        y = p.forward(X[100:105].contiguous(), q, s, z)
    size = X[100:105].double().abs() @ held.double().abs().t()
    u = U[dt]
    within(y, Y[100:105].double(), (u + 2 * K * E) * size + 2.1 * u * Y[100:105].double().abs(), "4-bit against dequantised")


@pytest.mark.parametrize("T,K", [(4, 512), (40, 8192)])
def test_streams_graphs_and_shared_plans(T, K):
    """One plan serves two weights; a captured call follows new rows."""
    N, G, dt = 264, 64, torch.bfloat16
    sets = [weights(N, K, G, dt, i, True, True, 2) for i in (1, 2)]
    packed = [w4_pack(rowmajor(c), s, z) for c, s, z in sets]
    X = ints((T, K), 2, gen(3), dt)
    p = W4Plan(T, N, K, dt, "GATED", group=G, act="RELU")

    def ref(i):
        y = [X.double() @ values(sets[i][0][m], sets[i][1][m], sets[i][2][m], G).t() for m in (0, 1)]
        return (y[0].clamp(min=0) * y[1])

    outs = [p.forward(X, *w) for w in packed]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = p.forward(X, *packed[0], stream=s)
    s.synchronize()
    assert torch.equal(side, outs[0])
    Y = torch.zeros((T, N), dtype=dt, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.gemm_epi_w4_execute(X, *packed[1], None, Y)
    for seed in (5, 6):
        X.copy_(ints((T, K), 2, gen(seed), dt))
        graph.replay()
        again = p.forward(X, *packed[1])
        torch.cuda.synchronize()
        assert torch.equal(Y, again)
        r = ref(1)
        # gate and up are exact; their product and its rounding: (u + 2 e) |H|
        within(Y, r, (U[dt] + 2 * E) * r.abs() + TINY[dt], "gated")


@pytest.mark.parametrize("gated", [False, True])
def test_shared_tiles(gated, monkeypatch):
    """Tiles cut at any block among 1 to 37 CTAs."""
    T, N, K, G, dt = 20, 400, 1408, 64, torch.bfloat16
    codes, s, z = weights(N, K, G, dt, 4, True, True, 2 if gated else None)
    w4 = w4_pack(rowmajor(codes), s, z)
    X = ints((T, K), 3, gen(4), dt)
    y = X.double() @ values(codes, s, z, G).reshape(-1, K).t()
    for grid in (1, 2, 3, 7, 12, 37):
        monkeypatch.setenv("GEMM_EPI_SKINNY_GRID", str(grid))
        with W4Plan(T, N, K, dt, "GATED" if gated else "NONE", group=G, act="RELU", out_f32=True) as p:
            assert p.info()["grid"] == grid
            Y = p.forward(X, *w4)
            for _ in range(3):
                assert torch.equal(Y, p.forward(X, *w4))
            assert p.status() == 0
        if gated:
            r = y[:, :N].clamp(min=0) * y[:, N:]
            within(Y, r, 2 * E * r.abs(), "gated")  # one fp32 product of exact sums
        else:
            assert torch.equal(Y.double(), y)


def test_watchdog_reports_and_the_plan_recovers(monkeypatch):
    T, N, K, G, dt = 20, 400, 1408, 64, torch.bfloat16
    codes, s, z = weights(N, K, G, dt, 4, True, True)
    w4 = w4_pack(rowmajor(codes), s, z)
    X = ints((T, K), 3, gen(4), dt)
    monkeypatch.setenv("GEMM_EPI_WAIT_TIMEOUT_MS", "50")
    monkeypatch.setenv("GEMM_EPI_TEST_HOOKS", "1")
    monkeypatch.setenv("GEMM_EPI_INJECT_STALL", "1")
    with W4Plan(T, N, K, dt, "NONE", group=G) as p:
        p.forward(X, *w4)
        torch.cuda.synchronize()
        assert p.status() == binding.ERR_TIMEOUT and p.status() == 0
    monkeypatch.delenv("GEMM_EPI_INJECT_STALL")
    with W4Plan(T, N, K, dt, "NONE", group=G, out_f32=True) as p:
        Y = p.forward(X, *w4)
        torch.cuda.synchronize()
        assert p.status() == 0
    assert torch.equal(Y.double(), X.double() @ values(codes, s, z, G).t())


def test_refusals():
    N, K, G, dt = 64, 256, 64, torch.bfloat16
    W = torch.zeros((N, K), dtype=dt, device="cuda")
    q, s, z = w4_quantize(W, group=G, zeros=True)
    X, Y = torch.zeros((4, K), dtype=dt, device="cuda"), torch.zeros((4, N), dtype=dt, device="cuda")
    with W4Plan(4, N, K, dt, "BIAS", group=G) as p, Plan(4, N, K, dt, "NONE") as d:
        with pytest.raises(GemmEpiError):  # no bias
            p.gemm_epi_w4_execute(X, q, s, z, None, Y)
        L = binding.lib()
        assert L.gemm_epi_w4_execute(d.handle, 32, 32, 32, None, None, 32, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_execute(p.handle, 32, 32, 32, 32, None, None) == binding.ERR_EPILOG_MISMATCH
        bias = torch.zeros(N, dtype=dt, device="cuda")
        assert L.gemm_epi_w4_execute(p.handle, X.data_ptr(), q.data_ptr() + 8, s.data_ptr(), None, bias.data_ptr(), Y.data_ptr(),
                                     None) == binding.ERR_MISALIGNED
        for bad in ((X.float(), q, s, z, bias, Y), (X, q[1:], s, z, bias, Y), (X, q, s.float(), z, bias, Y), (X, q, s, z[1:], bias, Y),
                    (X, q, s, z, bias[1:], Y), (X.cpu(), q, s, z, bias, Y)):
            with pytest.raises(ValueError):
                p.gemm_epi_w4_execute(*bad)
    for call in (lambda: gemm_epi_w4_quantize(W.float(), q, s, z, group=G), lambda: gemm_epi_w4_quantize(W, q, s.half(), z, group=G),
                 lambda: gemm_epi_w4_quantize(W, q[1:], s, z, group=G), lambda: gemm_epi_w4_quantize(W.t(), q, s, z, group=G),
                 lambda: gemm_epi_w4_dequantize(q, s, z, W.half(), group=G),
                 lambda: gemm_epi_w4_pack(W.to(torch.uint8), s.view(N, -1)[:, :2].contiguous(), None, q, s, z)):
        with pytest.raises((ValueError, GemmEpiError)):
            call()
