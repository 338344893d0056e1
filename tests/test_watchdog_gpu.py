"""The watchdog bounds waits, not launches.

A healthy launch that lasts several times the limit of one wait must end well:
every wait that can span many pipeline steps (the end of a CTA pair's second
CTA, the zeroing of an expert's foreign rows, a tile's accumulator) counts its
limit from the last step that was made. Whole-number inputs, so sampled rows
are exact.
"""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import GroupedPlan, MxPlan, Plan

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LIMIT_MS = 2


def signs(shape, seed):
    """-1, 0 or 1, as bf16."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).to(BF)


def limit(monkeypatch):
    monkeypatch.setenv("GEMM_EPI_WAIT_TIMEOUT_MS", str(LIMIT_MS))


def run_long(p, call):
    """Runs it and sees that it lasted more than twice the limit and that no wait ran out."""
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    call()
    b.record()
    torch.cuda.synchronize()
    assert p.status() == 0
    assert a.elapsed_time(b) > 2 * LIMIT_MS


def test_one_product_on_cta_pairs(monkeypatch):
    limit(monkeypatch)
    monkeypatch.setenv("GEMM_EPI_FORCE_KERNEL", "pair")
    T, N, K = 32768, 16384, 16384
    X, W = signs((T, K), 1), signs((K, N), 2)
    Y = torch.zeros((T, N), dtype=BF, device="cuda")
    with Plan(T, N, K, BF, "NONE") as p:
        assert p.info()["kernel"] == 2
        run_long(p, lambda: p.gemm_epi_execute(X, W, None, Y))
    for r in (slice(0, 3), slice(T - 3, T)):
        assert torch.equal(Y[r], (X[r].double() @ W.double()).to(BF))


@pytest.mark.parametrize("tr", [128, 256])
def test_grouped_forward(monkeypatch, tr):
    limit(monkeypatch)
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    T, N, K = 32768, 16384, 16384
    off = [0, 15001, T]
    X, W = signs((T, K), 1), signs((2, K, N), 2)
    Y = torch.zeros((T, N), dtype=BF, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    with GroupedPlan(2, T, N, K, BF, "NONE") as p:
        run_long(p, lambda: p.gemm_epi_grouped_execute(X, W, None, offsets, Y))
    for e, r in ((0, slice(0, 3)), (0, slice(14999, 15001)), (1, slice(15001, 15003)), (1, slice(T - 3, T))):
        assert torch.equal(Y[r], (X[r].double() @ W[e].double()).to(BF))


@pytest.mark.parametrize("tr", [128, 256])
def test_wgrad_whose_last_expert_alone_is_ragged(monkeypatch, tr):
    limit(monkeypatch)
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    sizes, K, N = (65536, 45), 8192, 8192
    T = sum(sizes)
    X, dZ = signs((T, K), 1), signs((T, N), 2)
    dW = torch.zeros((2, K, N), device="cuda")
    offsets = torch.tensor([0, sizes[0], T], dtype=torch.int32, device="cuda")
    with GroupedPlan(2, T, N, K, BF, "WGRAD", out_f32=True) as p:
        run_long(p, lambda: p.gemm_epi_grouped_wgrad_execute(X, dZ, offsets, dW))
    assert torch.equal(dW[0, :64].double(), X[:sizes[0], :64].double().t() @ dZ[:sizes[0]].double())
    assert torch.equal(dW[0, -64:].double(), X[:sizes[0], -64:].double().t() @ dZ[:sizes[0]].double())
    assert torch.equal(dW[1].double(), X[sizes[0]:].double().t() @ dZ[sizes[0]:].double())


@pytest.mark.parametrize("tr", [128, 256])
def test_wgrad_with_many_experts_to_clear_between_others(monkeypatch, tr):
    """The epilogue clears 34 GB while the products of the experts behind wait for it."""
    limit(monkeypatch)
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    E, K, N, rows = 1024, 2048, 4096, 40
    sizes = [rows] * 2 + [0] * (E - 7) + [rows] * 5
    T = sum(sizes)
    X, dZ = signs((T, K), 1), signs((T, N), 2)
    dW = torch.full((E, K, N), 77.0, device="cuda")
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
    with GroupedPlan(E, T, N, K, BF, "WGRAD", out_f32=True) as p:
        run_long(p, lambda: p.gemm_epi_grouped_wgrad_execute(X, dZ, offsets, dW))
    full = [0, 1] + list(range(E - 5, E))
    for i, e in enumerate(full):
        r = slice(rows * i, rows * (i + 1))
        assert torch.equal(dW[e].double(), X[r].double().t() @ dZ[r].double())
    assert not bool(dW[2:E - 5].any())


@pytest.mark.parametrize("tr", [128, 256])
def test_microscaled(monkeypatch, tr):
    limit(monkeypatch)
    monkeypatch.setenv("GEMM_EPI_FORCE_GROUPED", str(tr))
    T, N, K = 65536, 16384, 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    Xq = torch.randint(0, 256, (T, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    Wq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    lv = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
    lv = torch.cat([lv, -lv])
    Y = torch.zeros((T, N), dtype=BF, device="cuda")
    with MxPlan(T, N, K, BF, "NONE") as p:
        Xs = torch.full((p.x_scales,), 127, dtype=torch.uint8, device="cuda")  # all scales are 1
        Ws = torch.full((p.w_scales,), 127, dtype=torch.uint8, device="cuda")
        run_long(p, lambda: p.gemm_epi_mx_execute(Xq, Xs, Wq, Ws, None, Y))

    def values(q):
        return torch.stack([lv[(q & 15).long()], lv[(q >> 4).long()]], -1).flatten(-2)

    W = values(Wq[:512])
    for r in (slice(0, 3), slice(T - 3, T)):
        assert torch.equal(Y[r, :512], (values(Xq[r]) @ W.t()).to(BF))
