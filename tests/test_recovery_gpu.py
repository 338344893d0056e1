"""A plan whose kernel gave up a wait computes right results again afterwards.

One CTA of the first launch withholds a completion signal, so some parts of a
shared tile, or some row tiles of an expert, are counted in and others are not.
The report is read while the legacy stream is behind, and the next call runs on
a stream that does not wait for that one: the counts must be back at zero for
it all the same, and the inputs are others (parts of the interrupted launch
would show). Whole numbers, so sums are exact.
"""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GemmEpiError, GroupedPlan, MxPlan, binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def ints(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(BF)


@pytest.fixture
def stall(monkeypatch):
    monkeypatch.setenv("GEMM_EPI_TEST_HOOKS", "1")
    monkeypatch.setenv("GEMM_EPI_INJECT_STALL", "2")  # one CTA, the first launch only
    monkeypatch.setenv("GEMM_EPI_WAIT_TIMEOUT_MS", "50")
    return monkeypatch


def recover(p, call, check, read_by_call=False):
    s = torch.cuda.Stream()
    call(None, 0)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # the legacy stream is behind
    if read_by_call:
        with pytest.raises(GemmEpiError) as e:
            call(s, 1)
        assert e.value.code == binding.ERR_TIMEOUT
    else:
        assert p.status() == binding.ERR_TIMEOUT
    for _ in range(3):
        call(s, 1)
        s.synchronize()
        assert p.status() == 0
        check()


@pytest.mark.parametrize("read_by_call", [False, True])
@pytest.mark.parametrize("tr", [32, 128])
def test_shared_tiles(stall, tr, read_by_call):
    stall.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    stall.setenv("GEMM_EPI_FORCE_SPLIT", "4")
    T, N, K = 60, 264, 2048
    Xs, W = (ints((T, K), 3), ints((T, K), 1)), ints((2, K, N), 2)
    X = Xs[1]
    offsets = torch.tensor([0, 25, T], dtype=torch.int32, device="cuda")
    ref = torch.cat([X[:25].double() @ W[0].double(), X[25:].double() @ W[1].double()])
    Y = torch.zeros((T, N), device="cuda")
    with GroupedPlan(2, T, N, K, BF, "NONE", out_f32=True) as p:
        recover(p, lambda s, i: p.gemm_epi_grouped_execute(Xs[i], W, None, offsets, Y, stream=s),
                lambda: Y.double().equal(ref) or pytest.fail("Y"), read_by_call)


@pytest.mark.parametrize("tr,split", [(32, 1), (32, 4), (128, 1), (128, 4), (256, 1)])
def test_bias_gradient_of_several_row_tiles(stall, tr, split):
    stall.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    stall.setenv("GEMM_EPI_FORCE_SPLIT", str(split))
    T, N, K = 900, 136, 1024
    off = [0, 620, T]
    Xs, W = (ints((T, K), 3), ints((T, K), 1)), ints((2, K, N), 2)
    X = Xs[1]
    aux = torch.full((T, (N + 31) // 32), -1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    ref = torch.cat([X[:620].double() @ W[0].double(), X[620:].double() @ W[1].double()])
    db_ref = torch.stack([ref[:620].sum(0), ref[620:].sum(0)])
    dZ, db = torch.zeros((T, N), device="cuda"), torch.zeros((2, N), device="cuda")

    def check():
        assert torch.equal(dZ.double(), ref) and torch.equal(db.double(), db_ref)

    with GroupedPlan(2, T, N, K, BF, "DRELU_BGRAD", out_f32=True) as p:
        recover(p, lambda s, i: p.gemm_epi_grouped_drelu_bgrad_execute(Xs[i], W, aux, offsets, dZ, db, s), check)


@pytest.mark.parametrize("tr,split", [(128, 1), (128, 4), (256, 1)])
def test_wgrad(stall, tr, split):
    stall.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    stall.setenv("GEMM_EPI_FORCE_SPLIT", str(split))
    T, N, K = 1500, 136, 72
    Xs, dY = (ints((T, K), 3), ints((T, K), 1)), ints((T, N), 2)
    X = Xs[1]
    offsets = torch.tensor([0, 1027, T], dtype=torch.int32, device="cuda")
    ref = torch.stack([X[a:b].double().t() @ dY[a:b].double() for a, b in ((0, 1027), (1027, T))])
    db_ref = torch.stack([X[:1027].double().sum(0), X[1027:].double().sum(0)])
    dW, db = torch.zeros((2, K, N), device="cuda"), torch.zeros((2, K), device="cuda")

    def check():
        assert torch.equal(dW.double(), ref) and torch.equal(db.double(), db_ref)

    with GroupedPlan(2, T, N, K, BF, "WGRAD", out_f32=True) as p:
        recover(p, lambda s, i: p.gemm_epi_grouped_wgrad_execute(Xs[i], dY, offsets, dW, db, s), check)


@pytest.mark.parametrize("tr", [128, 256])
def test_microscaled(stall, tr):
    stall.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    T, N, K = 300, 264, 512
    xx, w = (ints((T, K), 3), ints((T, K), 1)), ints((N, K), 2)
    x = xx[1]
    q = [binding.mx_quantize(v) for v in xx]
    wq, ws = binding.mx_quantize(w)
    ref = x.double() @ w.double().t()
    Y = torch.zeros((T, N), device="cuda")
    with MxPlan(T, N, K, BF, "NONE", out_f32=True) as p:
        recover(p, lambda s, i: p.gemm_epi_mx_execute(*q[i], wq, ws, None, Y, stream=s),
                lambda: Y.double().equal(ref) or pytest.fail("Y"))
