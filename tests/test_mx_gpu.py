"""The microscaled 4-bit path on the GPU against its definition in 64 bits.

Quantisation has one right answer for every bit: the scale is a power of two,
x / scale is exact, and the rounding is stated; so bytes are compared. The
product of values whose scales lie within a factor of four is a sum of
multiples of 2^-4 below 2^24 of them, exact in fp32: Y is the exact result
rounded once, and compared with equality. Wide scales: the fp32 sum errs by at
most 2 K 2^-24 S (S the sum of |products|; 2 for a truncating adder), then the
bias's addition and one rounding, u |Y| (u = 2^-8, 2^-11, 2^-24).
"""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import (GemmEpiError, GroupedPlan, MxPlan, binding, gemm_epi_mx_dequantize,
                                         gemm_epi_mx_quantize, mx_quantize, mx_scales_bytes)

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ref_quantize(x):
    """[rows, cols] -> (values, codes, scale bytes) by the definition, in 64 bits."""
    R, C = x.shape
    b = x.double().view(R, C // 32, 32)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(top)
    pw = torch.tensor([2.0 ** i for i in range(-200, 200)], dtype=torch.float64, device="cuda")
    at = torch.searchsorted(pw, torch.where(bad, 1.0, top).contiguous(), right=True) - 1  # floor(log2 top) + 200
    byte = torch.where(top > 0, (at - 200 - 2 + 127).clamp(min=0), 0)
    byte = torch.where(bad, 255, byte)
    scale = pw[byte.clamp(max=254) - 127 + 200]
    y = (torch.where(bad[..., None], 0.0, b) / scale[..., None])
    lv = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    d = (y.abs()[..., None] - lv).abs()
    near = d == d.amin(-1, keepdim=True)
    even = torch.arange(8, device="cuda") % 2 == 0
    pick = torch.where(near.sum(-1, keepdim=True) > 1, near & even, near)
    code = pick.to(torch.uint8).argmax(-1)
    val = torch.where(y < 0, -lv[code], lv[code]) * scale[..., None]
    val = torch.where(bad[..., None], float("nan"), val)
    return val.view(R, C), (code + 8 * torch.signbit(y)).view(R, C), byte


def scale_bytes(s, row_tile, C, rows):
    """Scale bytes [rows, C / 32] read from the stated layout, starting at a tile of rows."""
    kt = -(-C // 128)
    r = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(C // 32, device="cuda")[None, :]
    return s[((row_tile + r // 128) * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4]


def spread(shape, g, dt, width=4.0):
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp(width * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    return x.clamp(-6e4, 6e4).to(dt)


def check_quantized(x, q, s, row_tile=0):
    val, code, byte = ref_quantize(x)
    R, C = x.shape
    got = torch.stack([q & 15, q >> 4], -1).view(R, C)
    finite = (byte != 255).repeat_interleave(32, 1)
    assert torch.equal(scale_bytes(s, row_tile, C, R).long(), byte)
    # the sign of a zero is free
    same = (got.long() == code) | ((got & 7) == 0) & ((code & 7) == 0)
    assert bool((same | ~finite).all())
    return val


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,C", [(1, 32), (3, 96), (129, 128), (70, 1120), (257, 2080), (1000, 64)])
def test_quantize_and_back(R, C, dtype):
    dt = DT[dtype]
    x = spread((R, C), gen(R + C), dt)
    x[R // 2, :32] = 0
    q, s = mx_quantize(x)
    val = check_quantized(x, q, s)
    for out_dt in (torch.float32, torch.bfloat16, torch.float16):
        out = torch.empty((R, C), dtype=out_dt, device="cuda")
        gemm_epi_mx_dequantize(q, s, out)
        assert torch.equal(out, val.to(out_dt))
    # blocks past the last column are written as zero
    kt = -(-C // 128)
    if C % 128:
        r = torch.arange(R, device="cuda")
        for b in range(C % 128 // 32, 4):
            assert bool((s[(r // 128 * kt + kt - 1) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_value_of_the_type(dtype):
    """All 65536 bit patterns, each in a block whose largest magnitude it shares with powers of two."""
    x = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(DT[dtype]).view(2048, 32)
    q, s = mx_quantize(x)
    check_quantized(x, q, s)
    y = x[torch.isfinite(x.float()).all(1)].clone()
    y[:, 0] = torch.where(torch.arange(len(y), device="cuda") % 2 == 0, 6.0, 4.0).to(y.dtype)  # one scale, all ties
    check_quantized(y, *mx_quantize(y))


def test_halfway_values_round_to_even_codes():
    x = torch.tensor([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 7.9] + [0] * 16,
                     dtype=torch.bfloat16, device="cuda")[None]
    out = torch.empty((1, 32), device="cuda")
    q, s = mx_quantize(x)
    gemm_epi_mx_dequantize(q, s, out)
    assert out[0, :16].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, 6]


def test_infinities_and_nans_stay_in_their_block():
    x = torch.randn((4, 128), generator=gen(3), device="cuda").bfloat16()
    x[0, 5], x[1, 40], x[2, 127] = float("inf"), float("nan"), float("-inf")
    q, s = mx_quantize(x)
    out = torch.empty((4, 128), device="cuda")
    gemm_epi_mx_dequantize(q, s, out)
    bad = torch.zeros((4, 4), dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 1] = bad[2, 3] = True
    assert torch.equal(torch.isnan(out).view(4, 4, 32).all(-1), bad) and torch.equal(torch.isnan(out).view(4, 4, 32).any(-1), bad)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,R,C", [(1, 8, 32), (2, 136, 160), (3, 72, 2080), (1, 1000, 416)])
def test_transposed_source(B, R, C, dtype):
    x = spread((B, R, C), gen(R), DT[dtype])
    q, s = mx_quantize(x)
    qt, st = mx_quantize(x.transpose(1, 2).contiguous(), transposed=True)
    for b in range(B):
        check_quantized(x[b], q[b], s, row_tile=b * (-(-R // 128)))
        check_quantized(x[b], qt[b], st, row_tile=b * (-(-R // 128)))


def test_grouped_rows_and_rows_of_no_group():
    sizes, front, behind, C = [0, 1, 130, 128, 0, 3, 260], 2, 4, 160
    off = [front]
    for n in sizes:
        off.append(off[-1] + n)
    T = off[-1] + behind
    x = spread((T, C), gen(7), torch.bfloat16)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    q = torch.full((T, C // 2), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((mx_scales_bytes(T, C, groups=len(sizes)),), 0x5A, dtype=torch.uint8, device="cuda")
    gemm_epi_mx_quantize(x, q, s, offsets=offsets)
    tile = 0
    out = torch.full((T, C), 77.0, device="cuda")
    gemm_epi_mx_dequantize(q, s, out, offsets=offsets)
    for e, n in enumerate(sizes):
        r = slice(off[e], off[e + 1])
        if n:
            val = check_quantized(x[r], q[r], s, row_tile=tile)
            assert torch.equal(out[r].double(), val)
        tile += -(-n // 128)
    for rows in (slice(0, front), slice(off[-1], T)):
        assert bool((q[rows] == 0x5A).all()) and bool((out[rows] == 77).all())


def random_mx(shape, g, lo=126, hi=128, fill=0xFF):
    """Random codes and scales of [batch, rows, cols], scale bytes of absent rows NaN (0xFF)."""
    B, R, C = shape
    q = torch.randint(0, 256, (B, R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    byte = torch.randint(lo, hi + 1, (B, R, C // 32), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((mx_scales_bytes(R, C, batch=B),), fill, dtype=torch.uint8, device="cuda")
    place(s, byte, [b * (-(-R // 128)) for b in range(B)], C)
    return q, s, decode(q, byte)


def place(s, byte, tiles, C):
    kt = -(-C // 128)
    for by, t in zip(byte, tiles):
        R = by.shape[0]
        r = torch.arange(R, device="cuda")[:, None]
        b = torch.arange(kt * 4, device="cuda")[None, :]
        full = torch.nn.functional.pad(by, (0, kt * 4 - by.shape[1]))
        s[((t + r // 128) * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = full


def decode(q, byte):
    lv = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device="cuda")
    v = torch.stack([lv[(q & 15).long()], lv[(q >> 4).long()]], -1).flatten(-2)
    pw = torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=torch.float64, device="cuda")
    return v * pw[byte.long()].repeat_interleave(32, -1)


def force(monkeypatch, tr):
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))


def epilog_of(Z, epilog):
    if epilog == "RELU_BIAS":
        return Z.clamp(min=0)
    return 0.5 * Z * (1 + torch.erf(Z / 2 ** 0.5)) if epilog == "GELU_BIAS" else Z


@pytest.mark.parametrize("tr", [128, 256])
@pytest.mark.parametrize("T,N,K", [(1, 8, 32), (5, 72, 64), (40, 200, 96), (129, 136, 288), (300, 520, 1056), (257, 256, 512)])
@pytest.mark.parametrize("epilog", ["NONE", "BIAS", "RELU_BIAS", "GELU_BIAS"])
def test_product(monkeypatch, epilog, T, N, K, tr):
    force(monkeypatch, tr)
    g = gen(T + N)
    Xq, Xs, X = random_mx((1, T, K), g)
    Wq, Ws, W = random_mx((1, N, K), g)
    dt = torch.bfloat16 if T % 2 else torch.float16
    b = torch.randint(-8, 9, (N,), generator=g, device="cuda").to(dt)
    for out_f32 in (False, True):
        with MxPlan(T, N, K, dt, epilog, out_f32=out_f32) as p:
            buf = torch.full((T * N + 512,), 77, dtype=p.out_dtype, device="cuda")
            Y = buf[256:-256].view(T, N)
            p.gemm_epi_mx_execute(Xq[0], Xs, Wq[0], Ws, None if epilog == "NONE" else b, Y)
            torch.cuda.synchronize()
            assert p.status() == 0
        assert bool((buf[:256] == 77).all()) and bool((buf[-256:] == 77).all())
        Z = X[0] @ W[0].t() + (0 if epilog == "NONE" else b.double())
        ref = epilog_of(Z, epilog)
        if epilog == "GELU_BIAS":
            assert bool(((Y.double() - ref).abs() <= U[Y.dtype] * ref.abs() + 2e-7 * Z.abs() + 1e-30).all())
        else:
            assert torch.equal(Y, ref.to(Y.dtype))


@pytest.mark.parametrize("tr", [128, 256])
@pytest.mark.parametrize("sizes,front,behind", [([0, 1, 17, 130, 0, 300, 2], 3, 5), ([5], 0, 0), ([0, 0], 1, 1),
                                                ([(11 * i) % 37 for i in range(70)], 0, 2), ([128, 256, 129], 0, 0)])
def test_grouped_product(monkeypatch, sizes, front, behind, tr):
    force(monkeypatch, tr)
    N, K, E = 200, 160, len(sizes)
    off = [front]
    for n in sizes:
        off.append(off[-1] + n)
    T = off[-1] + behind
    g = gen(T)
    Xq = torch.randint(0, 256, (T, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    byte = torch.randint(126, 129, (T, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    Xs = torch.full((mx_scales_bytes(T, K, groups=E),), 0xFF, dtype=torch.uint8, device="cuda")
    tile = 0
    for e, n in enumerate(sizes):
        place(Xs, [byte[off[e]:off[e + 1]]], [tile], K)
        tile += -(-n // 128)
    X = decode(Xq, byte)
    Wq, Ws, W = random_mx((E, N, K), g)
    b = torch.randint(-8, 9, (E, N), generator=g, device="cuda").bfloat16()
    with MxPlan(T, N, K, torch.bfloat16, "RELU_BIAS", E=E) as p:
        Y = torch.full((T, N), 77, dtype=torch.bfloat16, device="cuda")
        p.gemm_epi_mx_execute(Xq, Xs, Wq, Ws, b, Y, torch.tensor(off, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert p.status() == 0
    ref = torch.full((T, N), 77.0, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(off[e], off[e + 1])
        ref[r] = (X[r] @ W[e].t() + b[e].double()).clamp(min=0)
    assert torch.equal(Y, ref.to(torch.bfloat16))


@pytest.mark.parametrize("tr", [128, 256])
def test_wide_scales(monkeypatch, tr):
    force(monkeypatch, tr)
    T, N, K = 200, 264, 1056
    g = gen(5)
    Xq, Xs, X = random_mx((1, T, K), g, 100, 140)
    Wq, Ws, W = random_mx((1, N, K), g, 110, 130)
    with MxPlan(T, N, K, torch.bfloat16, "NONE", out_f32=True) as p:
        Y = p.forward(Xq[0], Xs, Wq[0], Ws, None)
    S = X[0].abs() @ W[0].abs().t()
    assert bool(((Y.double() - X[0] @ W[0].t()).abs() <= (2 * K + 1) * 2.0 ** -24 * S).all())


def test_nan_scale_reaches_only_its_row():
    T, N, K = 40, 72, 96
    g = gen(6)
    Xq, Xs, X = random_mx((1, T, K), g)
    Wq, Ws, W = random_mx((1, N, K), g)
    Xs[7 * 16 + 1] = 255  # row 7, block 1
    with MxPlan(T, N, K, torch.bfloat16, "NONE", out_f32=True) as p:
        Y = p.forward(Xq[0], Xs, Wq[0], Ws, None)
    assert bool(torch.isnan(Y[7]).all())
    keep = torch.arange(T, device="cuda") != 7
    assert torch.equal(Y[keep].double(), (X[0] @ W[0].t())[keep])


@pytest.mark.parametrize("grouped", [False, True])
def test_block_of_quantised_layers(grouped):
    """norm'd rows -> 4 bits -> product with ReLU -> 4 bits -> product, dense and by expert, against
    the definition chained in 64 bits on the values that each step really stored."""
    dt = torch.bfloat16
    sizes = [30, 0, 150, 1] if grouped else [181]
    off = [0]
    for n in sizes:
        off.append(off[-1] + n)
    T, D, F, E = off[-1], 160, 288, len(sizes)
    g = gen(8)
    X = torch.randn((T, D), generator=g, device="cuda").to(dt)
    W1 = (torch.randn((E, D, F), generator=g, device="cuda") / D ** 0.5).to(dt)   # K x N, as this library's weights
    W2 = (torch.randn((E, D, F), generator=g, device="cuda") / F ** 0.5).to(dt)   # N x K, [out, in]
    b1, b2 = torch.randn((E, F), generator=g, device="cuda").to(dt), torch.randn((E, D), generator=g, device="cuda").to(dt)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda") if grouped else None
    W1q, W1s = mx_quantize(W1, transposed=True)
    W2q, W2s = mx_quantize(W2)
    with MxPlan(T, F, D, dt, "RELU_BIAS", E=E if grouped else None) as up, \
            MxPlan(T, D, F, dt, "BIAS", E=E if grouped else None, out_f32=True) as down:
        Xq, Xs = mx_quantize(X, offsets)
        H = up.forward(Xq, Xs, W1q, W1s, b1, offsets)
        Hq, Hs = mx_quantize(H, offsets)
        Y = down.forward(Hq, Hs, W2q, W2s, b2, offsets)
        torch.cuda.synchronize()
        assert up.status() == 0 and down.status() == 0
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        x, w1, w2 = ref_quantize(X[r])[0], ref_quantize(W1[e].t().contiguous())[0], ref_quantize(W2[e])[0]
        Z = x @ w1.t() + b1[e].double()
        S = x.abs() @ w1.abs().t() + b1[e].double().abs()
        assert bool(((H[r].double() - Z.clamp(min=0)).abs() <= 2 * (D + 1) * 2.0 ** -24 * S + U[dt] * Z.abs()).all())
        h = ref_quantize(H[r])[0]
        S = h.abs() @ w2.abs().t() + b2[e].double().abs()
        assert bool(((Y[r].double() - (h @ w2.t() + b2[e].double())).abs() <= (2 * (F + 1) + 1) * 2.0 ** -24 * S).all())


def test_captured_and_other_stream():
    T, N, K = 64, 200, 160
    g = gen(9)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    Wq, Ws, W = random_mx((1, N, K), g)
    q = torch.zeros((T, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.zeros(mx_scales_bytes(T, K), dtype=torch.uint8, device="cuda")
    with MxPlan(T, N, K, torch.bfloat16, "NONE") as p:
        Y = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            gemm_epi_mx_quantize(x, q, s)
            p.gemm_epi_mx_execute(q, s, Wq[0], Ws, None, Y)
        for seed in (1, 2):
            x.copy_(torch.randn((T, K), generator=gen(seed), device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            got = Y.clone()
            st.wait_stream(torch.cuda.current_stream())
            gemm_epi_mx_quantize(x, q, s, stream=st)
            p.gemm_epi_mx_execute(q, s, Wq[0], Ws, None, Y, stream=st)
            torch.cuda.synchronize()
            assert p.status() == 0 and torch.equal(got, Y)
            ref = ref_quantize(x)[0] @ W[0].t()
            S = ref_quantize(x)[0].abs() @ W[0].abs().t()
            assert bool(((Y.double() - ref).abs() <= 2 * K * 2.0 ** -24 * S + U[torch.bfloat16] * ref.abs()).all())


def test_sizes_past_32_bit_offsets():
    """More than 2^31 elements quantised, given back, and written by the product."""
    R, C = 33000, 65536
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    x[:3] = spread((3, C), gen(1), torch.bfloat16)
    x[-2:] = spread((2, C), gen(2), torch.bfloat16)
    q, s = mx_quantize(x)
    val = ref_quantize(x[-2:])
    assert torch.equal(torch.stack([q[-2:] & 7, q[-2:] >> 4 & 7], -1).view(2, C).long(), val[1] & 7)
    out = torch.empty((R, C), dtype=torch.bfloat16, device="cuda")
    gemm_epi_mx_dequantize(q, s, out)
    assert torch.equal(out[-2:], val[0].to(torch.bfloat16)) and torch.equal(out[:3], ref_quantize(x[:3])[0].to(torch.bfloat16))
    assert bool((out[3:-2] == 0).all())
    del x, q, s, out
    T, N, K = 270000, 8192, 32
    g = gen(3)
    Xq, Xs, X = random_mx((1, T, K), g)
    Wq, Ws, W = random_mx((1, N, K), g)
    with MxPlan(T, N, K, torch.bfloat16, "NONE") as p:
        Y = p.forward(Xq[0], Xs, Wq[0], Ws, None)
        torch.cuda.synchronize()
        assert p.status() == 0
    for rows in (slice(0, 5), slice(T - 300, T)):
        assert torch.equal(Y[rows], (X[0, rows] @ W[0].t()).to(torch.bfloat16))


def test_refusals_on_a_live_plan():
    L = binding.lib()
    x = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda").data_ptr()
    q = x.data_ptr()
    with MxPlan(64, 64, 64, torch.bfloat16, "BIAS") as d, MxPlan(64, 64, 64, torch.bfloat16, "BIAS", E=2) as e, \
            GroupedPlan(2, 64, 64, 64, torch.bfloat16, "BIAS") as gp:
        assert L.gemm_epi_mx_execute(d.handle, q, q, q, q, q, o, q, None) == binding.ERR_INVALID_ARG
        assert L.gemm_epi_mx_execute(e.handle, q, q, q, q, q, None, q, None) == binding.ERR_INVALID_ARG
        assert L.gemm_epi_mx_execute(d.handle, q, q + 4, q, q, q, None, q, None) == binding.ERR_MISALIGNED
        assert L.gemm_epi_mx_execute(d.handle, q, q, q, q, None, None, q, None) == binding.ERR_INVALID_ARG
        assert L.gemm_epi_mx_execute(gp.handle, q, q, q, q, q, o, q, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_execute(d.handle, q, q, q, q, None, None) == binding.ERR_EPILOG_MISMATCH
        assert d.info()["kernel"] == 6 and d.info()["tile_k"] == 256
        with pytest.raises(ValueError):
            d.gemm_epi_mx_execute(x, x, x, x, None, x)
    with pytest.raises(ValueError):
        gemm_epi_mx_quantize(torch.zeros((4, 64), device="cuda"), x, x)
    with pytest.raises(GemmEpiError):
        MxPlan(64, 64, 64, torch.bfloat16, "RELU_AUX_BIAS")


@pytest.mark.parametrize("tr", [128, 256])
def test_watchdog(monkeypatch, tr):
    force(monkeypatch, tr)
    monkeypatch.setenv("GEMM_EPI_TEST_HOOKS", "1")
    monkeypatch.setenv("GEMM_EPI_INJECT_STALL", "1")
    monkeypatch.setenv("GEMM_EPI_WAIT_TIMEOUT_MS", "50")
    g = gen(14)
    Xq, Xs, _ = random_mx((1, 64, 64), g)
    Wq, Ws, _ = random_mx((1, 64, 64), g)
    with MxPlan(64, 64, 64, torch.bfloat16, "NONE") as p:
        p.forward(Xq[0], Xs, Wq[0], Ws, None)
        torch.cuda.synchronize()
        assert p.status() == binding.ERR_TIMEOUT
        assert p.status() == 0
