"""Outputs of the conveniences belong to the stream that the call runs on.

The current stream is behind, and the memory that it has just given back is
still to be written by work that waits there. A convenience called on another
stream must not take that memory for an output: its kernel ends first, and the
late writes would land in a finished result. Integer inputs, so every result is
exact.

A plan's counters are zero before its first call, whatever stream that runs on.
"""
import ctypes

import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GroupedPlan, MxPlan, Plan, binding, mx_quantize

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
T, N, K = 520, 264, 136


def ints(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(BF)


class Behind:
    """The current stream works for some milliseconds, then overwrites blocks that are free by then."""

    def __init__(self):
        self.busy = torch.randn((4096, 4096), device="cuda")

    def __call__(self, *outputs):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        late = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in outputs]
        for _ in range(8):
            self.busy = self.busy @ self.busy * 1e-3
        for x in late:
            x.fill_(77)


def streams():
    s = torch.cuda.Stream()
    return (s, s.cuda_stream)


def test_one_product():
    behind = Behind()
    X, W, dZ, b = ints((T, K), 1), ints((K, N), 2), ints((T, N), 3), ints((N,), 4)
    Z = X.double() @ W.double() + b.double()
    G = X.double() @ W.double()
    aux = torch.full((T, (N + 31) // 32), -1, dtype=torch.int32, device="cuda")
    for s in streams():
        with Plan(T, N, K, BF, "GELU_AUX_BIAS") as p:
            behind(((T, N), BF), ((T, N), BF))
            _, z = p.forward(X, W, b, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(z, Z.to(BF))
        with Plan(T, N, K, BF, "BIAS") as p:
            behind(((T, N), BF))
            Y, _ = p.forward(X, W, b, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(Y, Z.to(BF))
        with Plan(T, N, K, BF, "DRELU_BGRAD") as p:
            behind(((T, N), BF), ((N,), torch.float32))
            dX, db = p.backward(X, W, aux, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(dX, G.to(BF)) and torch.equal(db.double(), G.sum(0))
        with Plan(T, N, K, BF, "WGRAD") as p:
            behind(((K, N), BF), ((K,), torch.float32))
            dW, db = p.wgrad(X, dZ, with_dbias=True, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(dW, (X.double().t() @ dZ.double()).to(BF)) and torch.equal(db.double(), X.double().sum(0))


def test_grouped():
    behind = Behind()
    off = [0, 300, 300, T - 3]
    E = len(off) - 1
    X, W, dZ = ints((T, K), 1), ints((E, K, N), 2), ints((T, N), 3)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    aux = torch.full((T, (N + 31) // 32), -1, dtype=torch.int32, device="cuda")
    G = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    dW_ref = torch.zeros((E, K, N), dtype=torch.float64, device="cuda")
    db_ref, dx_ref = torch.zeros((E, N), dtype=torch.float64, device="cuda"), torch.zeros((E, K), dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(off[e], off[e + 1])
        G[r] = X[r].double() @ W[e].double()
        db_ref[e], dx_ref[e] = G[r].sum(0), X[r].double().sum(0)
        dW_ref[e] = X[r].double().t() @ dZ[r].double()
    for s in streams():
        with GroupedPlan(E, T, N, K, BF, "NONE") as p:
            behind(((T, N), BF))
            Y, _ = p.forward(X, W, None, offsets, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(Y, G.to(BF))
        with GroupedPlan(E, T, N, K, BF, "DRELU_BGRAD") as p:
            behind(((T, N), BF), ((E, N), torch.float32))
            dX, db = p.backward(X, W, aux, offsets, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(dX, G.to(BF)) and torch.equal(db.double(), db_ref)
        for out_f32 in (False, True):
            with GroupedPlan(E, T, N, K, BF, "WGRAD", out_f32=out_f32) as p:
                behind(((E, K, N), p.out_dtype), ((E, K), torch.float32))
                dW, db = p.wgrad(X, dZ, offsets, with_dbias=True, stream=s)
                torch.cuda.synchronize()
                assert torch.equal(dW, dW_ref.to(dW.dtype)) and torch.equal(db.double(), dx_ref)


def test_microscaled():
    behind = Behind()
    rows, cols = 200, 160
    # whole numbers up to 3 are held exactly (scale 1/2 or 1/4)
    x, w = ints((rows, cols), 5), ints((72, cols), 6)
    for s in streams():
        behind(((rows, cols // 2), torch.uint8))
        xq, xs = mx_quantize(x, stream=s)
        wq, ws = mx_quantize(w, stream=s)
        with MxPlan(rows, 72, cols, BF, "NONE", out_f32=True) as p:
            behind(((rows, 72), torch.float32))
            Y = p.forward(xq, xs, wq, ws, None, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(Y.double(), x.double() @ w.double().t())


def test_handle_zero_is_the_legacy_stream():
    """The outputs of a call on stream handle 0 belong to the legacy stream, which that handle means."""
    X, W = ints((T, K), 1), ints((1, K, N), 2)
    offsets = torch.tensor([0, T - 9], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        with binding._on_stream(0, X.device):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
        with GroupedPlan(1, T, N, K, BF, "NONE") as p:
            torch.cuda._sleep(100_000_000)
            Y, _ = p.forward(X, W, None, offsets, stream=0)
            torch.cuda.synchronize()
    assert torch.equal(Y[:T - 9], (X[:T - 9].double() @ W[0].double()).to(BF)) and not bool(Y[T - 9:].any())


def dirty_small_blocks():
    """Device memory that small allocations are likely to get next, filled with ones."""
    rt = ctypes.CDLL("libcudart.so.12")
    blocks = [ctypes.c_void_p() for _ in range(256)]
    for b in blocks:
        assert rt.cudaMalloc(ctypes.byref(b), ctypes.c_size_t(4096)) == 0
        assert rt.cudaMemset(b, 0xFF, ctypes.c_size_t(4096)) == 0
    torch.cuda.synchronize()
    for b in blocks:
        assert rt.cudaFree(b) == 0


def test_a_new_plan_on_a_stream_of_its_own(monkeypatch):
    """Made while the legacy stream is behind, and run at once on a stream that does not wait for it."""
    s = torch.cuda.Stream()
    R, K1, N1 = 300, 2048, 264
    X, W = ints((R, K1), 1), ints((1, K1, N1), 2)
    Y = torch.zeros((R, N1), device="cuda")
    G = X.double() @ W[0].double()
    aux = torch.full((R, (N1 + 31) // 32), -1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    db = torch.zeros((1, N1), device="cuda")
    few, Yf = ints((40, K1), 3), torch.zeros((40, N1), device="cuda")
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", "128")
    monkeypatch.setenv("GEMM_EPI_FORCE_SPLIT", "4")

    def grouped():
        with GroupedPlan(1, R, N1, K1, BF, "DRELU_BGRAD", out_f32=True) as p:
            p.gemm_epi_grouped_drelu_bgrad_execute(X, W, aux, offsets, Y, db, stream=s)
            s.synchronize()
        assert torch.equal(Y.double(), G) and torch.equal(db[0].double(), G.sum(0))

    def one():
        with Plan(R, N1, K1, BF, "DRELU_BGRAD", out_f32=True) as p:
            p.drelu_bgrad_execute(X, W[0], aux, Y, db[0], stream=s)
            s.synchronize()
        assert torch.equal(Y.double(), G) and torch.equal(db[0].double(), G.sum(0))

    def few_rows():
        with Plan(40, N1, K1, BF, "NONE", out_f32=True) as p:
            assert p.info()["split_k"] > 1
            p.gemm_epi_execute(few, W[0], None, Yf, stream=s)
            s.synchronize()
        assert torch.equal(Yf.double(), few.double() @ W[0].double())

    for run in (grouped, one, few_rows):
        Y.zero_()
        db.zero_()
        dirty_small_blocks()
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)
        run()
        torch.cuda.synchronize()
