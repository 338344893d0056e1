"""Expert-grouped products on the GPU against a plain loop over the experts in
64 bits.

Integer inputs in [-3, 3]: every product and fp32 partial sum is an exact
small integer (|Z| <= 9 K + 3 < 2^24), so Y, the mask, dZ, dbias and dW have
one right value each -- the exact one, rounded once to the output type -- and
the comparison is equality. GELU's bound: u |Y| for the rounding to the 16-bit
output (u = half a step, 2^-8 or 2^-11) plus 2e-7 |Z| for erff and the fp32
products around it (a few units of 2^-24 relative to |Z|). Normal inputs: the
fp32 dot product errs by at most 2 K 2^-24 S (S the sum of |products|; 2 for a
truncating adder), then one rounding.

Rows outside every expert hold NaN in X, and the weights of experts without
rows are NaN: neither may show in any output.
"""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GemmEpiError, GroupedPlan, Plan, binding

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
NAN = float("nan")

# rows per expert, rows in front of the first and behind the last
LAYOUTS = {"mixed": ([0, 1, 17, 33, 0, 129, 300, 2], 0, 5), "single": ([1], 0, 0), "one": ([77], 3, 4),
           "large": ([513, 0, 260], 0, 0), "empty": ([0, 0, 0], 2, 6),
           "many": ([(7 * i) % 23 for i in range(150)], 1, 1)}
SHAPES = [(200, 136), (72, 24), (264, 520), (8, 8)]  # N, K


def offsets_of(sizes, front):
    o = [front]
    for s in sizes:
        o.append(o[-1] + s)
    return o


def ints(shape, lo, hi, g, dt):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(dt)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def outside_nan(x, off):
    x = x.clone()
    x[:off[0]] = NAN
    x[off[-1]:] = NAN
    return x


def bits_of(words, N):
    w = words.to(torch.int64) & 0xFFFFFFFF
    return (((w[:, :, None] >> torch.arange(32, device="cuda")) & 1) != 0).reshape(words.shape[0], -1)[:, :N]


def guarded(shape, dtype):
    """Sentinel-filled output inside a larger buffer."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 512,), 77, dtype=dtype, device="cuda")
    return buf, buf[256:256 + n].view(shape)


def guards_ok(buf):
    return bool((buf[:256] == 77).all()) and bool((buf[-256:] == 77).all())


def force(monkeypatch, tr):
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))


def make(layout, N, K, dt, seed=1):
    sizes, front, behind = LAYOUTS[layout]
    off = offsets_of(sizes, front)
    T = off[-1] + behind
    g = gen(seed)
    X = outside_nan(ints((T, K), -3, 3, g, dt), off)
    W = ints((len(sizes), K, N), -3, 3, g, dt)
    b = ints((len(sizes), N), -3, 3, g, dt)
    for e, s in enumerate(sizes):
        if s == 0:
            W[e] = NAN
    return sizes, off, T, X, W, b


def check_forward(layout, N, K, dt, epilog, w_nk=False, out_f32=False, bias_f32=False, stream=None):
    sizes, off, T, X, W, b = make(layout, N, K, dt)
    E = len(sizes)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    with GroupedPlan(E, T, N, K, dt, epilog, w_nk=w_nk, out_f32=out_f32) as p:
        if bias_f32:
            p.set_bias_f32(True)
        ybuf, Y = guarded((T, N), p.out_dtype)
        spec = p.aux_spec()
        abuf, aux = guarded(*spec) if spec else (None, None)
        p.gemm_epi_grouped_execute(X, W.transpose(1, 2).contiguous() if w_nk else W, b.float() if bias_f32 else b,
                                   offsets, Y, aux, stream)
        torch.cuda.synchronize()
        assert p.status() == 0
    assert guards_ok(ybuf) and (abuf is None or guards_ok(abuf))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if sizes[e] == 0:
            continue
        Z = X[r].double() @ W[e].double()
        if epilog != "NONE":
            Z = Z + b[e].double()
        if epilog.startswith("GELU"):
            ref = 0.5 * Z * (1 + torch.erf(Z / 2 ** 0.5))
            assert bool(((Y[r].double() - ref).abs() <= U[Y.dtype] * ref.abs() + 2e-7 * Z.abs() + 1e-30).all())
            if epilog == "GELU_AUX_BIAS":
                assert torch.equal(aux[r], Z.to(dt))
        else:
            ref = Z.clamp(min=0) if epilog.startswith("RELU") else Z
            assert torch.equal(Y[r], ref.to(Y.dtype)), f"expert {e}"
            if epilog == "RELU_AUX_BIAS":
                assert torch.equal(bits_of(aux[r], N), Z > 0)
                if N % 32:
                    assert bool(((aux[r, -1].to(torch.int64) & 0xFFFFFFFF) >> (N % 32) == 0).all())
    for out in (Y, aux):
        if out is not None:
            assert bool((out[:off[0]] == 77).all()) and bool((out[off[-1]:] == 77).all()), "rows of no expert changed"


@pytest.mark.parametrize("tr", [32, 128, 256])
@pytest.mark.parametrize("w_nk", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("epilog", ["NONE", "BIAS", "RELU_BIAS", "RELU_AUX_BIAS", "GELU_BIAS", "GELU_AUX_BIAS"])
def test_forward(monkeypatch, epilog, dtype, w_nk, tr):
    force(monkeypatch, tr)
    check_forward("mixed", 200, 136, DT[dtype], epilog, w_nk=w_nk)


@pytest.mark.parametrize("tr", [32, 128, 256])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_forward_layouts(monkeypatch, layout, N, K, tr):
    force(monkeypatch, tr)
    check_forward(layout, N, K, torch.bfloat16, "RELU_AUX_BIAS")


@pytest.mark.parametrize("tr", [32, 128, 256])
def test_forward_fp32_output_and_bias(monkeypatch, tr):
    force(monkeypatch, tr)
    check_forward("mixed", 72, 264, torch.float16, "RELU_AUX_BIAS", out_f32=True, bias_f32=True)
    check_forward("mixed", 136, 72, torch.bfloat16, "GELU_AUX_BIAS", w_nk=True, out_f32=True)


def check_backward(layout, N, K, dt, w_nk=False, out_f32=False):
    sizes, off, T, dY, W, _ = make(layout, N, K, dt, seed=3)
    E = len(sizes)
    words = (N + 31) // 32
    aux = torch.randint(-2 ** 31, 2 ** 31, (T, words), generator=gen(5), device="cuda").to(torch.int32)
    if N % 32:
        aux[:, -1] &= (1 << (N % 32)) - 1
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    W2 = W.transpose(1, 2).contiguous() if w_nk else W
    with GroupedPlan(E, T, N, K, dt, "DRELU_BGRAD", w_nk=w_nk, out_f32=out_f32) as p:
        for _ in range(2):  # the tickets are back at zero for the second call
            zbuf, dZ = guarded((T, N), p.out_dtype)
            bbuf, db = guarded((E, N), torch.float32)
            p.gemm_epi_grouped_drelu_bgrad_execute(dY, W2, aux, offsets, dZ, db)
            torch.cuda.synchronize()
            assert p.status() == 0
            assert guards_ok(zbuf) and guards_ok(bbuf)
            for e in range(E):
                r = slice(off[e], off[e + 1])
                if sizes[e] == 0:
                    assert bool((db[e] == 0).all())
                    continue
                G = torch.where(bits_of(aux[r], N), dY[r].double() @ W[e].double(), 0.0)
                assert torch.equal(dZ[r], G.to(dZ.dtype)), f"expert {e}"
                assert torch.equal(db[e].double(), G.sum(0)), f"expert {e}"
            assert bool((dZ[:off[0]] == 77).all()) and bool((dZ[off[-1]:] == 77).all())


@pytest.mark.parametrize("tr", [32, 128, 256])
@pytest.mark.parametrize("w_nk", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_backward(monkeypatch, dtype, w_nk, tr):
    force(monkeypatch, tr)
    check_backward("mixed", 200, 136, DT[dtype], w_nk=w_nk)


@pytest.mark.parametrize("tr", [32, 128, 256])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_backward_layouts(monkeypatch, layout, N, K, tr):
    force(monkeypatch, tr)
    check_backward(layout, N, K, torch.bfloat16, out_f32=layout == "large")


def check_wgrad(layout, N, K, dt, out_f32=False, with_dbias=True):
    sizes, off, T, X, _, _ = make(layout, N, K, dt, seed=7)
    E = len(sizes)
    dZ = outside_nan(ints((T, N), -3, 3, gen(8), dt), off)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    with GroupedPlan(E, T, N, K, dt, "WGRAD", out_f32=out_f32) as p:
        wbuf, dW = guarded((E, K, N), p.out_dtype)
        bbuf, db = guarded((E, K), torch.float32)
        p.gemm_epi_grouped_wgrad_execute(X, dZ, offsets, dW, db if with_dbias else None)
        torch.cuda.synchronize()
        assert p.status() == 0
    assert guards_ok(wbuf) and guards_ok(bbuf)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        ref = X[r].double().t() @ dZ[r].double()
        assert torch.equal(dW[e], ref.to(dW.dtype)), f"expert {e}"
        if with_dbias:
            assert torch.equal(db[e].double(), X[r].double().sum(0))


@pytest.mark.parametrize("tr", [128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("out_f32", [False, True])
def test_wgrad(monkeypatch, dtype, out_f32, tr):
    force(monkeypatch, tr)
    check_wgrad("mixed", 200, 136, DT[dtype], out_f32=out_f32)


@pytest.mark.parametrize("tr", [128, 256])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_wgrad_layouts(monkeypatch, layout, N, K, tr):
    force(monkeypatch, tr)
    check_wgrad(layout, N, K, torch.bfloat16, with_dbias=layout != "large")


@pytest.mark.parametrize("split", [1, 2, 5, 16])
@pytest.mark.parametrize("tr", [32, 128])
@pytest.mark.parametrize("layout", ["mixed", "single", "empty", "large"])
def test_split_contraction(monkeypatch, layout, tr, split):
    """Tiles whose contraction several CTAs share, more parts than k-blocks among them."""
    force(monkeypatch, tr)
    monkeypatch.setenv("GEMM_EPI_FORCE_SPLIT", str(split))
    for epilog in ("RELU_AUX_BIAS", "GELU_AUX_BIAS", "NONE"):
        check_forward(layout, 72, 264, torch.bfloat16, epilog, w_nk=split == 2, out_f32=split == 5)
    check_backward(layout, 200, 520, torch.bfloat16)
    if tr == 128:
        check_wgrad(layout, 72, 136, torch.bfloat16, out_f32=split == 5)


def test_few_tiles_over_a_long_contraction():
    """The kernel's own choice of the split: one narrow expert, and one long one beside a short one."""
    g = gen(21)
    T, N, K = 5, 64, 4096
    X, W = ints((T, K), -1, 1, g, torch.bfloat16), ints((1, K, N), -1, 1, g, torch.bfloat16)
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    aux = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    with GroupedPlan(1, T, N, K, torch.bfloat16, "DRELU_BGRAD", out_f32=True) as p:
        for _ in range(3):
            dZ, db = p.backward(X, W, aux, offsets)
            ref = X.double() @ W[0].double()
            assert torch.equal(dZ.double(), ref) and torch.equal(db[0].double(), ref.sum(0))
    X, dZ = ints((3005, 40), -1, 1, g, torch.bfloat16), ints((3005, 72), -1, 1, g, torch.bfloat16)
    offsets = torch.tensor([0, 2999, 2999, 3005], dtype=torch.int32, device="cuda")
    with GroupedPlan(3, 3005, 72, 40, torch.bfloat16, "WGRAD", out_f32=True) as p:
        for _ in range(2):
            dW, db = p.wgrad(X, dZ, offsets, with_dbias=True)
            for e, (a, b) in enumerate(((0, 2999), (2999, 2999), (2999, 3005))):
                assert torch.equal(dW[e].double(), X[a:b].double().t() @ dZ[a:b].double())
                assert torch.equal(db[e].double(), X[a:b].double().sum(0))


@pytest.mark.parametrize("tail", list(range(1, 17)) + [47, 48, 49, 63, 64, 65])
def test_wgrad_row_tails_keep_foreign_rows_out(monkeypatch, tail):
    """Every length of an expert's last k-block, with NaN right behind it."""
    g = gen(tail)
    X, dZ = ints((tail + 70, 136), -3, 3, g, torch.bfloat16), ints((tail + 70, 200), -3, 3, g, torch.bfloat16)
    X[tail:], dZ[tail:] = NAN, NAN
    offsets = torch.tensor([0, tail], dtype=torch.int32, device="cuda")
    for tr in (128, 256):
        force(monkeypatch, tr)
        with GroupedPlan(1, tail + 70, 200, 136, torch.bfloat16, "WGRAD") as p:
            dW = p.wgrad(X, dZ, offsets)
            torch.cuda.synchronize()
            assert p.status() == 0
        assert torch.equal(dW[0], (X[:tail].double().t() @ dZ[:tail].double()).to(torch.bfloat16))


@pytest.mark.parametrize("tr", [32, 128, 256])
def test_normal_inputs(monkeypatch, tr):
    force(monkeypatch, tr)
    sizes, off, T, _, _, _ = make("mixed", 264, 1032, torch.float16)
    g = gen(11)
    K, N, E = 1032, 264, len(sizes)
    X = torch.randn((T, K), generator=g, device="cuda").half()
    W = (torch.randn((E, K, N), generator=g, device="cuda") / K ** 0.5).half()
    b = torch.randn((E, N), generator=g, device="cuda").half()
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    with GroupedPlan(E, T, N, K, torch.float16, "BIAS", out_f32=True) as p:
        Y, _ = p.forward(X, W, b, offsets)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        S = X[r].double().abs() @ W[e].double().abs() + b[e].double().abs()
        err = (Y[r].double() - (X[r].double() @ W[e].double() + b[e].double())).abs()
        assert bool((err <= 2 * (K + 1) * 2.0 ** -24 * S).all())


@pytest.mark.parametrize("bad", [[0, 40, 20, 60], [-5, 10, 30, 30], [0, 10, 1000, 2000], [50, 40, 30, 20], [7, 7, 7, 2 ** 31 - 1]])
@pytest.mark.parametrize("tr", [32, 128, 256])
def test_offsets_are_cut_to_the_rows(monkeypatch, bad, tr):
    """Decreasing or outlying offsets name the rows of their running maximum cut to [0, T]."""
    force(monkeypatch, tr)
    T, N, K = 60, 72, 40
    off, m = [], 0
    for v in bad:
        m = max(m, min(max(v, 0), T))
        off.append(m)
    g = gen(2)
    X, W = ints((T, K), -3, 3, g, torch.bfloat16), ints((3, K, N), -3, 3, g, torch.bfloat16)
    offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
    with GroupedPlan(3, T, N, K, torch.bfloat16, "NONE") as p:
        buf, Y = guarded((T, N), torch.bfloat16)
        p.gemm_epi_grouped_execute(X, W, None, offsets, Y)
        torch.cuda.synchronize()
    assert guards_ok(buf)
    ref = torch.full((T, N), 77.0, dtype=torch.float64, device="cuda")
    for e in range(3):
        ref[off[e]:off[e + 1]] = X[off[e]:off[e + 1]].double() @ W[e].double()
    assert torch.equal(Y, ref.to(torch.bfloat16))


def test_one_expert_equals_one_product():
    T, N, K = 300, 200, 136
    g = gen(4)
    X, W, b = ints((T, K), -3, 3, g, torch.bfloat16), ints((K, N), -3, 3, g, torch.bfloat16), ints((N,), -3, 3, g, torch.bfloat16)
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    with Plan(T, N, K, torch.bfloat16, "RELU_AUX_BIAS") as p, GroupedPlan(1, T, N, K, torch.bfloat16, "RELU_AUX_BIAS") as q:
        Y, aux = p.forward(X, W, b)
        Yg, auxg = q.forward(X, W[None], b[None], offsets)
    assert torch.equal(Y, Yg) and torch.equal(aux, auxg)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_expert_block_step_against_autograd(dtype):
    """A whole two-layer expert block, forward and backward, weights [out, in],
    chained through the mask, against 64-bit autograd; small integers, exact."""
    dt = DT[dtype]
    sizes = [0, 3, 130, 1, 40]
    off = offsets_of(sizes, 0)
    E, T, D, F = len(sizes), off[-1], 72, 136
    g = gen(6)
    X, dY = ints((T, D), -1, 1, g, dt), ints((T, D), -1, 1, g, dt)
    W1, b1 = ints((E, F, D), -1, 1, g, dt), ints((E, F), -2, 2, g, dt)
    W2, b2 = ints((E, D, F), -1, 1, g, dt), ints((E, D), -2, 2, g, dt)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    with GroupedPlan(E, T, F, D, dt, "RELU_AUX_BIAS", w_nk=True) as up, \
            GroupedPlan(E, T, D, F, dt, "BIAS", w_nk=True) as down, \
            GroupedPlan(E, T, F, D, dt, "DRELU_BGRAD") as dup, \
            GroupedPlan(E, T, F, D, dt, "WGRAD", out_f32=True) as w2g, \
            GroupedPlan(E, T, D, F, dt, "WGRAD", out_f32=True) as w1g, \
            GroupedPlan(E, T, D, F, dt, "NONE") as dx:
        H, aux = up.forward(X, W1, b1, offsets)
        Y, _ = down.forward(H, W2, b2, offsets)
        dZ1, db1 = dup.backward(dY, W2, aux, offsets)
        dW2, db2 = w2g.wgrad(dY, H, offsets, with_dbias=True)
        dW1 = w1g.wgrad(dZ1, X, offsets)
        dX, _ = dx.forward(dZ1, W1, None, offsets)
        torch.cuda.synchronize()
    P = [t.double().requires_grad_() for t in (X, W1, b1, W2, b2)]
    Yr = torch.cat([torch.relu(P[0][off[e]:off[e + 1]] @ P[1][e].t() + P[2][e]) @ P[3][e].t() + P[4][e] for e in range(E)])
    Yr.backward(dY.double())
    assert float(Yr.detach().abs().max()) <= 256 and float(P[0].grad.abs().max()) <= 256  # exact in 16 bits
    assert torch.equal(Y.double(), Yr.detach())
    for got, want in ((dX, P[0]), (dW1, P[1]), (db1, P[2]), (dW2, P[3]), (db2, P[4])):
        assert torch.equal(got.double(), want.grad)


def test_gradient_against_differences():
    """dX through the mask against central differences of the block's output, in 64 bits."""
    dt = torch.float16
    sizes, D, F = [2, 0, 3], 8, 16
    off = offsets_of(sizes, 0)
    g = gen(9)
    X, W1, b1 = ints((5, D), -3, 3, g, dt), ints((3, D, F), -3, 3, g, dt), ints((3, F), -3, 3, g, dt) + 0.5
    dH = ints((5, D), -3, 3, g, dt)  # gradient behind a second product with W2
    W2 = ints((3, D, F), -3, 3, g, dt)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    with GroupedPlan(3, 5, F, D, dt, "RELU_AUX_BIAS") as up, GroupedPlan(3, 5, F, D, dt, "DRELU_BGRAD") as back:
        _, aux = up.forward(X, W1, b1, offsets)
        dZ, db = back.backward(dH, W2, aux, offsets)

    def loss(b):
        return sum(((torch.relu(X[off[e]:off[e + 1]].double() @ W1[e].double() + b[e]) @ W2[e].double().t())
                    * dH[off[e]:off[e + 1]].double()).sum() for e in range(3))

    b = b1.double()  # half-integers: no pre-activation within 1/4 of zero, so the loss is linear around b
    for e in range(3):
        for j in range(F):
            d = torch.zeros_like(b)
            d[e, j] = 0.25
            diff = (loss(b + d) - loss(b - d)) / 0.5
            assert float(diff) == float(db[e, j])


def test_captured_call_follows_new_offsets():
    T, N, K, E = 100, 72, 136, 4
    g = gen(12)
    X, W = ints((T, K), -3, 3, g, torch.bfloat16), ints((E, K, N), -3, 3, g, torch.bfloat16)
    aux = torch.full((T, 3), -1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 25, 50, 75, 100], dtype=torch.int32, device="cuda")
    with GroupedPlan(E, T, N, K, torch.bfloat16, "DRELU_BGRAD") as p:
        dZ = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
        db = torch.zeros((E, N), device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            p.gemm_epi_grouped_drelu_bgrad_execute(X, W, aux, offsets, dZ, db)
        for off in ([0, 25, 50, 75, 100], [0, 0, 99, 99, 100], [10, 11, 12, 13, 14]):
            offsets.copy_(torch.tensor(off, dtype=torch.int32))
            dZ.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert p.status() == 0
            for e in range(E):
                G = X[off[e]:off[e + 1]].double() @ W[e].double()
                assert torch.equal(dZ[off[e]:off[e + 1]], G.to(torch.bfloat16)) and torch.equal(db[e].double(), G.sum(0))
            assert bool((dZ[:off[0]] == 7).all()) and bool((dZ[off[-1]:] == 7).all())


def test_other_stream_and_repeatability():
    sizes, off, T, X, W, b = make("large", 200, 136, torch.bfloat16)
    g = gen(13)
    X = torch.randn((T, 136), generator=g, device="cuda").bfloat16()
    W = torch.randn((3, 136, 200), generator=g, device="cuda").bfloat16()
    aux = torch.full((T, 7), -1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = []
    with GroupedPlan(3, T, 200, 136, torch.bfloat16, "DRELU_BGRAD") as p:
        for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
            dZ, db = torch.zeros((T, 200), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 200), device="cuda")
            torch.cuda.synchronize()
            p.gemm_epi_grouped_drelu_bgrad_execute(X, W, aux, offsets, dZ, db, stream)
            torch.cuda.synchronize()
            got.append((dZ, db))
    for dZ, db in got[1:]:
        assert torch.equal(dZ, got[0][0]) and torch.equal(db, got[0][1])


def test_gelu_of_special_values():
    """One term a product, so Z is the weight itself: infinities, NaN, far and near values."""
    z = torch.tensor([float("inf"), float("-inf"), NAN, 60000.0, -60000.0, 5.25, -5.25, 5.0, -5.0, 1.0, -1.0, 0.0, -0.0, 2.0 ** -24,
                      -(2.0 ** -24), 0.5], device="cuda").half()
    X = torch.zeros((3, 8), dtype=torch.float16, device="cuda")
    X[:, 0] = 1
    W = torch.zeros((1, 8, 16), dtype=torch.float16, device="cuda")
    W[0, 0] = z
    b = torch.zeros((1, 16), dtype=torch.float16, device="cuda")
    offsets = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    with GroupedPlan(1, 3, 16, 8, torch.float16, "GELU_BIAS", out_f32=True) as p:
        Y, _ = p.forward(X, W, b, offsets)
    d = z.double()
    ref = torch.where(d == float("-inf"), 0.0, d * torch.special.ndtr(d))
    assert bool((torch.isnan(Y) == torch.isnan(ref)).all()) and bool(torch.isinf(Y[:, 0]).all())
    fine = torch.isfinite(ref)
    assert bool(((Y[:, fine].double() - ref[fine]).abs() <= 2e-7 * d[fine].abs()).all())
    assert bool((Y[:, 1] == 0).all()) and bool((Y[:, 4] == 0).all())


def test_conveniences_on_another_stream():
    """The zeros that forward and backward start from are written on the call's stream."""
    g = gen(41)
    T, N, K = 4000, 1024, 64
    X, W = ints((T, K), -3, 3, g, torch.bfloat16), ints((2, K, N), -3, 3, g, torch.bfloat16)
    offsets = torch.tensor([0, 1500, T - 7], dtype=torch.int32, device="cuda")
    aux = torch.full((T, N // 32), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    ref[:1500], ref[1500:T - 7] = X[:1500].double() @ W[0].double(), X[1500:T - 7].double() @ W[1].double()
    busy = torch.randn((4096, 4096), device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with GroupedPlan(2, T, N, K, torch.bfloat16, "NONE") as p, GroupedPlan(2, T, N, K, torch.bfloat16, "DRELU_BGRAD") as q:
        for stream in (s, s.cuda_stream):
            for _ in range(8):
                busy = busy @ busy * 1e-3  # the current stream is behind
            Y, _ = p.forward(X, W, None, offsets, stream=stream)
            dZ, _ = q.backward(X, W, aux, offsets, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(Y, ref.to(torch.bfloat16)) and torch.equal(dZ, Y)


def test_two_plans_at_once():
    """Two plans on two streams, each with tickets and partials of its own, over and over."""
    g = gen(42)
    cases = []
    for T, N, K, E in ((3000, 520, 72, 3), (5, 64, 4096, 1)):
        X, W = ints((T, K), -1, 1, g, torch.bfloat16), ints((E, K, N), -1, 1, g, torch.bfloat16)
        offsets = torch.linspace(0, T, E + 1, device="cuda").to(torch.int32)
        off = offsets.tolist()
        aux = torch.full((T, (N + 31) // 32), -1, dtype=torch.int32, device="cuda")
        G = torch.cat([X[off[e]:off[e + 1]].double() @ W[e].double() for e in range(E)])
        db = torch.stack([G[off[e]:off[e + 1]].sum(0) for e in range(E)])
        p = GroupedPlan(E, T, N, K, torch.bfloat16, "DRELU_BGRAD", out_f32=True)
        out = torch.zeros((T, N), device="cuda"), torch.zeros((E, N), device="cuda")
        cases.append((p, X, W, aux, offsets, out, G, db, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for p, X, W, aux, offsets, out, _, _, s in cases:
            p.gemm_epi_grouped_drelu_bgrad_execute(X, W, aux, offsets, *out, s)
    torch.cuda.synchronize()
    for p, *_, out, G, db, _ in cases:
        assert p.status() == 0 and torch.equal(out[0].double(), G) and torch.equal(out[1].double(), db)
        p.free()


def test_bias_gradient_of_many_experts_without_rows(monkeypatch):
    E, T, N, K = 1000, 2, 2056, 16
    g = gen(43)
    X, W = ints((T, K), -3, 3, g, torch.bfloat16), ints((E, K, N), -3, 3, g, torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[501:] = 2
    aux = torch.full((T, (N + 31) // 32), -1, dtype=torch.int32, device="cuda")
    for tr in (32, 256):
        force(monkeypatch, tr)
        with GroupedPlan(E, T, N, K, torch.bfloat16, "DRELU_BGRAD") as p:
            db = torch.full((E, N), NAN, device="cuda")
            dZ = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
            p.gemm_epi_grouped_drelu_bgrad_execute(X, W, aux, off, dZ, db)
            ref = torch.zeros((E, N), dtype=torch.float64, device="cuda")
            ref[500] = (X.double() @ W[500].double()).sum(0)
            assert torch.equal(db.double(), ref) and p.info()["grid"] > 100


def test_refusals_on_a_live_plan():
    L = binding.lib()
    x = torch.zeros(64 * 64, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = x.data_ptr()
    with GroupedPlan(2, 64, 64, 64, torch.bfloat16, "RELU_AUX_BIAS") as p, \
            Plan(64, 64, 64, torch.bfloat16, "BIAS") as d, GroupedPlan(2, 64, 64, 64, torch.bfloat16, "DRELU_BGRAD") as bw:
        h, off = p.handle, o.data_ptr()
        assert L.gemm_epi_grouped_execute(h, q, q, q, None, q, q, None) == binding.ERR_INVALID_ARG
        assert L.gemm_epi_grouped_execute(h, q, q, q, off, q, None, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_grouped_execute(h, q + 8, q, q, off, q, q, None) == binding.ERR_MISALIGNED
        assert L.gemm_epi_grouped_execute(h, q, q, q, off + 2, q, q, None) == binding.ERR_MISALIGNED
        assert L.gemm_epi_grouped_execute(bw.handle, q, q, q, off, q, q, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_grouped_wgrad_execute(h, q, q, off, q, None, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_grouped_drelu_bgrad_execute(h, q, q, q, off, q, q, None) == binding.ERR_EPILOG_MISMATCH
        # a plan of one kind in the other kind's call
        assert L.gemm_epi_execute(h, q, q, q, q, q, None) == binding.ERR_EPILOG_MISMATCH
        assert L.gemm_epi_grouped_execute(d.handle, q, q, q, off, q, q, None) == binding.ERR_EPILOG_MISMATCH
        assert L.drelu_bgrad_execute(bw.handle, q, q, q, q, q, None) == binding.ERR_EPILOG_MISMATCH
        with pytest.raises(ValueError):
            p.gemm_epi_grouped_execute(x.view(64, 64), x, x, o, x)
        with pytest.raises(TypeError):
            p.gemm_epi_grouped_execute(None, x, x, o, x)
        with pytest.raises(GemmEpiError):  # a bias is missing
            p.gemm_epi_grouped_execute(x.view(64, 64), torch.zeros((2, 64, 64), dtype=torch.bfloat16, device="cuda"), None, o,
                                       x.view(64, 64), torch.zeros((64, 2), dtype=torch.int32, device="cuda"))
        info = p.info()
        assert (info["T"], info["N"], info["K"], info["kernel"], info["tile_n"]) == (64, 64, 64, 3, 32)
    with pytest.raises(GemmEpiError):
        GroupedPlan(2, 64, 60, 64, torch.bfloat16, "BIAS")


@pytest.mark.parametrize("tr", [32, 256])
def test_a_thousand_experts(monkeypatch, tr):
    force(monkeypatch, tr)
    g = gen(31)
    E, N, K = 1000, 40, 24
    sizes = torch.randint(0, 3, (E,), generator=g, device="cuda").tolist()
    sizes[517] = 300
    off = offsets_of(sizes, 0)
    T = off[-1]
    X, W = ints((T, K), -3, 3, g, torch.bfloat16), ints((E, K, N), -3, 3, g, torch.bfloat16)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(sizes, device="cuda"))
    ref = torch.bmm(X.double()[:, None], W.double()[e])[:, 0]
    with GroupedPlan(E, T, N, K, torch.bfloat16, "NONE") as p:
        Y, _ = p.forward(X, W, None, offsets)
    assert torch.equal(Y, ref.to(torch.bfloat16))
    dZ = ints((T, N), -3, 3, g, torch.bfloat16)
    with GroupedPlan(E, T, N, K, torch.bfloat16, "WGRAD", out_f32=True) as p:
        dW, db = p.wgrad(X, dZ, offsets, with_dbias=True)
    outer = torch.zeros((E, K, N), dtype=torch.float64, device="cuda").index_add_(0, e, X.double()[:, :, None] * dZ.double()[:, None])
    assert torch.equal(dW.double(), outer)
    assert torch.equal(db.double(), torch.zeros((E, K), dtype=torch.float64, device="cuda").index_add_(0, e, X.double()))


def test_outputs_past_32_bit_offsets():
    """More than 2^31 elements of Y, of the mask's rows, and of dW."""
    g = gen(32)
    T, N, K = 270000, 8192, 8
    X, W = ints((T, K), -3, 3, g, torch.bfloat16), ints((2, K, N), -3, 3, g, torch.bfloat16)
    b = ints((2, N), -3, 3, g, torch.bfloat16)
    offsets = torch.tensor([0, 5, T - 3], dtype=torch.int32, device="cuda")
    with GroupedPlan(2, T, N, K, torch.bfloat16, "RELU_AUX_BIAS") as p:
        Y, aux = p.forward(X, W, b, offsets)
        torch.cuda.synchronize()
        assert p.status() == 0
    for rows in (slice(5, 9), slice(T - 400, T - 3)):
        Z = X[rows].double() @ W[1].double() + b[1].double()
        assert torch.equal(Y[rows], Z.clamp(min=0).to(torch.bfloat16)) and torch.equal(bits_of(aux[rows], N), Z > 0)
    assert bool((Y[T - 3:] == 0).all())
    del Y, aux, X, W
    E, K = 34, 8192
    X, dZ = ints((E * 3, K), -3, 3, g, torch.bfloat16), ints((E * 3, N), -3, 3, g, torch.bfloat16)
    offsets = torch.arange(E + 1, device="cuda", dtype=torch.int32) * 3
    with GroupedPlan(E, E * 3, N, K, torch.bfloat16, "WGRAD") as p:
        dW = p.wgrad(X, dZ, offsets)
        torch.cuda.synchronize()
        assert p.status() == 0
    for e in (0, 32, 33):
        assert torch.equal(dW[e], (X[3 * e:3 * e + 3].double().t() @ dZ[3 * e:3 * e + 3].double()).to(torch.bfloat16))


@pytest.mark.parametrize("tr", [32, 256])
@pytest.mark.parametrize("split", [1, 4])
def test_watchdog(monkeypatch, tr, split):
    """A withheld completion signal ends the wait in time and is reported; the plan works again afterwards."""
    force(monkeypatch, tr)
    monkeypatch.setenv("GEMM_EPI_FORCE_SPLIT", str(split))
    monkeypatch.setenv("GEMM_EPI_TEST_HOOKS", "1")
    monkeypatch.setenv("GEMM_EPI_INJECT_STALL", "1")
    monkeypatch.setenv("GEMM_EPI_WAIT_TIMEOUT_MS", "50")
    g = gen(14)
    X, W = ints((64, 64), -3, 3, g, torch.bfloat16), ints((2, 64, 64), -3, 3, g, torch.bfloat16)
    offsets = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    with GroupedPlan(2, 64, 64, 64, torch.bfloat16, "NONE") as p:
        p.forward(X, W, None, offsets)
        torch.cuda.synchronize()
        assert p.status() == binding.ERR_TIMEOUT
        assert p.status() == 0
        with pytest.raises(GemmEpiError):  # the next call reports the run-out of the one before
            p.forward(X, W, None, offsets)
            torch.cuda.synchronize()
            p.forward(X, W, None, offsets)
