"""Cases of the expert (grouped) products and of the microscaled 4-bit path.

Five operators:

* ``forward``   grouped forward product: rows sorted by expert, one weight per
                expert, the framework's forward epilogs.
* ``backward``  grouped DRELU_BGRAD: the masked gradient and each expert's bias
                gradient.
* ``wgrad``     grouped weight gradient: a contraction over each expert's rows.
* ``mx_round``  4-bit microscaled quantisation and its inverse (what a
                calibration pass runs; what is held in 4 bits comes back as
                the values it stands for).
* ``mx_linear`` activations quantised on the fly, then the product with a
                weight held in 4 bits, dense or grouped by expert.

The plain forms gather each expert's rows into one padded batch and use torch
products in 32 bits. Operands of the 16-bit products lie on a fixed-point grid
(7 bits and a sign), as 8-bit checkpoints and activations give: every fp32 sum
is then exact, so the sign of a pre-activation, and with it the stored mask,
does not depend on the order of summation.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a small model: 8 token slots over 16 experts, latency only
        dict(name="forward decode", op="forward", dtype="bf16", E=16, T=8, K=2048, N=512, epilog="RELU_BIAS",
             w_nk=False, out_f32=False, skew=0.5, behind=0, split=1),
        # a serving batch of 64 slots over 8 experts: every weight streamed once, [out, in] checkpoints
        dict(name="forward serving", op="forward", dtype="bf16", E=8, T=64, K=4096, N=11008, epilog="GELU_BIAS",
             w_nk=True, out_f32=False, skew=0.5, behind=3, split=2),
        # a training step: 4096 tokens, two experts each, the mask kept for the backward
        dict(name="forward training", op="forward", dtype="bf16", E=8, T=8192, K=4096, N=11008, epilog="RELU_AUX_BIAS",
             w_nk=False, out_f32=False, skew=0.3, behind=0, split=3),
        # many small experts of odd sizes, ragged feature tiles
        dict(name="backward ragged", op="backward", dtype="fp16", E=64, T=4011, K=1024, N=5000, w_nk=True,
             out_f32=False, skew=0.8, behind=11, split=4),
        # the training step's backward product
        dict(name="backward training", op="backward", dtype="bf16", E=8, T=8192, K=4096, N=11008, w_nk=False,
             out_f32=False, skew=0.3, behind=0, split=5),
        # weight gradients kept in fp32 for an optimizer, with the second layer's bias gradient
        dict(name="wgrad ragged", op="wgrad", dtype="fp16", E=32, T=4011, K=1024, N=2048, out_f32=True, dbias=True,
             skew=0.8, behind=11, split=6),
        # the training step's weight gradient
        dict(name="wgrad training", op="wgrad", dtype="bf16", E=8, T=8192, K=4096, N=11008, out_f32=False, dbias=False,
             skew=0.3, behind=0, split=7),
        # a batch of activations, row by row
        dict(name="mx_round activations", op="mx_round", dtype="bf16", R=1000, C=4096, transposed=False),
        # a checkpoint's weight, given with the features contiguous
        dict(name="mx_round weight", op="mx_round", dtype="bf16", R=11008, C=4096, transposed=True),
        # one decoding step through a 4-bit layer
        dict(name="mx_linear decode", op="mx_linear", dtype="bf16", E=0, T=4, K=4096, N=11008, epilog="BIAS", skew=0.0,
             behind=0, split=8),
        # a prompt through a 4-bit layer
        dict(name="mx_linear prompt", op="mx_linear", dtype="bf16", E=0, T=4096, K=4096, N=11008, epilog="RELU_BIAS",
             skew=0.0, behind=0, split=9),
        # a serving batch through 4-bit experts of odd sizes
        dict(name="mx_linear experts", op="mx_linear", dtype="fp16", E=16, T=1003, K=2048, N=5000, epilog="GELU_BIAS",
             skew=0.6, behind=5, split=10),
    ]


def draw(rng):
    def size(lo, hi, step):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(v / step) * step)

    op = rng.choice(["forward", "forward", "backward", "wgrad", "mx_round", "mx_linear", "mx_linear"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "mx_round":
        transposed = rng.random() < 0.5
        return dict(op=op, dtype=dtype, R=size(8, 11008, 8) if transposed else size(1, 11008, 1),
                    C=size(32, 11008, 32), transposed=transposed)
    step = 32 if op == "mx_linear" else 8
    while True:
        E = rng.choice([0, 0, size(1, 64, 1)]) if op == "mx_linear" else size(1, 64, 1)
        T, K, N = size(1, 8192, 1), size(64, 8192, step), size(64, 11008, 8)
        if T * K * N <= 8192 * 4096 * 11008 and max(E, 1) * K * N <= 8 * 4096 * 11008:
            break
    c = dict(op=op, dtype=dtype, E=E, T=T, K=K, N=N, skew=rng.choice([0.0, 0.3, 0.8, 1.5]),
             behind=min(T - 1, rng.choice([0, 0, 1, 7])) if E else 0, split=rng.randrange(1 << 30))
    if op == "forward":
        c.update(epilog=rng.choice(["NONE", "BIAS", "RELU_BIAS", "RELU_AUX_BIAS", "GELU_BIAS", "GELU_AUX_BIAS"]),
                 w_nk=rng.random() < 0.5, out_f32=rng.random() < 0.2)
    elif op == "backward":
        c.update(w_nk=rng.random() < 0.5, out_f32=rng.random() < 0.2)
    elif op == "wgrad":
        c.update(out_f32=rng.random() < 0.3, dbias=rng.random() < 0.5)
    else:
        c.update(epilog=rng.choice(["NONE", "BIAS", "RELU_BIAS", "GELU_BIAS"]))
    return c


def group_sizes(case):
    """Rows per expert: a skewed multinomial draw (some experts get none)."""
    if not case["E"]:
        return np.array([case["T"]])
    r = np.random.RandomState(case["split"] % (1 << 31))
    w = np.exp(case["skew"] * r.randn(case["E"]))
    return r.multinomial(case["T"] - case["behind"], w / w.sum())


# -------------------------------------------------------------------- inputs
def _grid(shape, unit, g, dtype):
    """Normal draws rounded to a grid of `unit`, std 32 units, at most 127."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(32).round_().clamp_(-127, 127).mul_(unit).to(dtype)


def _swizzle(s):
    """Scale bytes [B, rows, blocks] -> the library's layout: tiles of 128 rows x 4 blocks,
    512 bytes each, row r at 16 (r % 32) + 4 (r / 32 % 4)."""
    B, R, C = s.shape
    s = torch.nn.functional.pad(s, (0, -C % 4, 0, -R % 128))
    return s.view(B, s.shape[1] // 128, 4, 32, s.shape[2] // 4, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(-1)


def _unswizzle(s, B, R, C):
    rt, kt = -(-R // 128), -(-C // 4)
    return s.view(B, rt, kt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(B, rt * 128, kt * 4)[:, :R, :C]


def _mx_weight(E, N, K, g):
    """A weight held in 4 bits: random codes and a narrow range of block scales."""
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    mid = 127 - round(math.log2(math.sqrt(K) * 2.7))
    s = torch.randint(mid - 1, mid + 2, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    return q, _swizzle(s)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case, "op": op, "dtype": dt}
    if op == "mx_round":
        R, C = case["R"], case["C"]
        # activations of very different rows and a few outliers, as norms leave them
        shape = (C, R) if case["transposed"] else (R, C)
        x = torch.randn(shape, generator=g, device="cuda")
        x *= torch.exp(2 * torch.randn((shape[0], 1), generator=g, device="cuda"))
        s["X"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 1e-3, x * 16, x).clamp_(-6e4, 6e4).to(dt)
        if own:
            from gemm_epilogues_tcgen05_b200 import binding

            s["q"] = torch.empty((R, C // 2), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(binding.mx_scales_bytes(R, C), dtype=torch.uint8, device="cuda")
            s["values"] = torch.empty((R, C), dtype=torch.float32, device="cuda")
        return s
    T, K, N, E = case["T"], case["K"], case["N"], max(case["E"], 1)
    sizes = group_sizes(case)
    sizes = sizes[np.random.RandomState(int(seed) % (1 << 31)).permutation(len(sizes))]
    off = np.concatenate([[0], np.cumsum(sizes)])
    s["sizes"] = sizes
    s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    # where each row goes in the plain form's padded batch
    rows, most = int(off[-1]), max(1, int(sizes.max()))
    expert = np.repeat(np.arange(len(sizes)), sizes)
    s["rows"], s["most"] = rows, most
    s["slot"] = torch.tensor(expert * most + np.arange(rows) - off[expert], dtype=torch.int64, device="cuda")
    if op == "mx_linear":
        s["X"] = torch.randn((T, K), generator=g, device="cuda").to(dt)
        s["Wq"], s["Ws"] = _mx_weight(E, N, K, g)
        s["bias"] = (torch.randn((E, N), generator=g, device="cuda") * 0.3).to(dt)
        s["Y"] = torch.zeros((T, N), dtype=dt, device="cuda")
        if own:
            from gemm_epilogues_tcgen05_b200 import binding

            s["plan"] = binding.MxPlan(T, N, K, dt, case["epilog"], E=case["E"] or None)
            s["Xq"] = torch.empty((T, K // 2), dtype=torch.uint8, device="cuda")
            s["Xs"] = torch.empty(binding.mx_scales_bytes(T, K, groups=case["E"] or None), dtype=torch.uint8,
                                  device="cuda")
        return s
    out = torch.float32 if case["out_f32"] else dt
    words = (N + 31) // 32
    if op == "wgrad":
        s["X"] = _grid((T, K), 2.0 ** -5, g, dt)
        dZ = _grid((T, N), 2.0 ** -7, g, dt)
        s["dZ"] = dZ * (torch.rand((T, N), generator=g, device="cuda") < 0.5)  # the ReLU's inactive half
        s["dW"] = torch.zeros((E, K, N), dtype=out, device="cuda")
        s["dbias"] = torch.zeros((E, K), dtype=torch.float32, device="cuda") if case["dbias"] else None
    else:
        unit = 2.0 ** -(5 + round(math.log2(math.sqrt(K))))
        s["X"] = _grid((T, K), 2.0 ** -5, g, dt)
        s["W"] = _grid((E, N, K) if case["w_nk"] else (E, K, N), unit, g, dt)
        if op == "forward":
            s["bias"] = _grid((E, N), 2.0 ** -7, g, dt)
            s["Y"] = torch.zeros((T, N), dtype=out, device="cuda")
            s["aux"] = (torch.zeros((T, words), dtype=torch.int32, device="cuda") if case["epilog"] == "RELU_AUX_BIAS"
                        else torch.zeros((T, N), dtype=dt, device="cuda") if case["epilog"] == "GELU_AUX_BIAS" else None)
        else:
            m = torch.randint(-2 ** 31, 2 ** 31, (T, words), generator=g, device="cuda").to(torch.int32)
            if N % 32:
                m[:, -1] &= (1 << (N % 32)) - 1
            s["aux"] = m
            s["dZ"] = torch.zeros((T, N), dtype=out, device="cuda")
            s["dbias"] = torch.zeros((E, N), dtype=torch.float32, device="cuda")
    if own:
        from gemm_epilogues_tcgen05_b200 import binding

        epi = {"forward": case.get("epilog"), "backward": "DRELU_BGRAD", "wgrad": "WGRAD"}[op]
        s["plan"] = binding.GroupedPlan(E, T, N, K, dt, epi, w_nk=case.get("w_nk", False), out_f32=case["out_f32"])
    return s


# --------------------------------------------------------------- plain forms
def _pad(s, X):
    """The rows of X in the padded batch [E, most, cols], fp32."""
    E = len(s["sizes"])
    P = torch.zeros((E * s["most"], X.shape[1]), dtype=torch.float32, device="cuda")
    P[s["slot"]] = X[:s["rows"]].float()
    return P.view(E, s["most"], X.shape[1])


def _unpad(s, P, dtype, T):
    Y = torch.zeros((T, P.shape[2]), dtype=dtype, device="cuda")
    Y[:s["rows"]] = P.view(-1, P.shape[2])[s["slot"]].to(dtype)
    return Y


def _pack(bits):
    """Truth values [T, N] -> 32-bit mask words, lowest column in the lowest bit."""
    T, N = bits.shape
    b = torch.nn.functional.pad(bits, (0, -N % 32)).view(T, -1, 32).to(torch.int64)
    return (b << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)


def _unpack(words, N):
    return (((words.to(torch.int64)[:, :, None] >> torch.arange(32, device="cuda")) & 1) != 0).view(words.shape[0], -1)[:, :N]


def _epilog(Z, epilog):
    if epilog.startswith("RELU"):
        return torch.where(Z > 0, Z, torch.zeros((), device="cuda"))
    if epilog.startswith("GELU"):
        return 0.5 * Z * (1 + torch.erf(Z * math.sqrt(0.5)))
    return Z


def _pow2(e):
    """2^e for whole e, exactly (a library power may be off in the last place, which moves ties)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64).float()


def _mx_values(x):
    """The values that x [rows, cols] stands for once held in microscaled 4 bits: blocks of 32
    along a row share the power of two 2^(floor(log2 max|x|) - 2); each element over it is
    rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, at most 6)."""
    b = x.float().view(x.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(top)
    e = torch.where(top > 0, e - 3, -127).clamp(min=-127)
    y = b * _pow2(-e)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    v = torch.tensor(E2M1, device="cuda")[code.long()]
    return (torch.where(y < 0, -v, v) * _pow2(e)).view(x.shape)


def _mx_decode(q, scales):
    """Packed codes [E, N, K/2] and their scales -> fp32 [E, N, K]."""
    E, N, K2 = q.shape
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = torch.stack([lut[(q & 15).long()], lut[(q >> 4).long()]], -1).view(E, N, K2 // 16, 32)
    e = _unswizzle(scales, E, N, K2 // 16).to(torch.int32) - 127
    return (v * _pow2(e[..., None])).view(E, N, 2 * K2)


def _plain(s):
    case, op, dt = s["case"], s["op"], s["dtype"]
    if op == "mx_round":
        return _mx_values(s["X"].t().contiguous() if case["transposed"] else s["X"])
    T, N = case["T"], case["N"]
    if op == "mx_linear":
        Z = torch.bmm(_pad(s, _mx_values(s["X"])), _mx_decode(s["Wq"], s["Ws"]).transpose(1, 2))
        if case["epilog"] != "NONE":
            Z = Z + s["bias"].float()[:, None]
        return _unpad(s, _epilog(Z, case["epilog"]), dt, T)
    out = torch.float32 if case["out_f32"] else dt
    if op == "wgrad":
        P = _pad(s, s["X"])
        dW = torch.bmm(P.transpose(1, 2), _pad(s, s["dZ"])).to(out)
        return {"dW": dW, "dbias": P.sum(1) if case["dbias"] else None}
    W = s["W"].float()
    Z = torch.bmm(_pad(s, s["X"]), W.transpose(1, 2) if case["w_nk"] else W)
    if op == "backward":
        Z = torch.where(_pad(s, _unpack(s["aux"], N)) != 0, Z, torch.zeros((), device="cuda"))
        return {"dZ": _unpad(s, Z, out, T), "dbias": Z.sum(1)}
    if case["epilog"] != "NONE":
        Z = Z + s["bias"].float()[:, None]
    Y = _unpad(s, _epilog(Z, case["epilog"]), out, T)
    if case["epilog"] == "RELU_AUX_BIAS":
        bits = torch.zeros((T, N), dtype=torch.bool, device="cuda")
        bits[:s["rows"]] = (Z > 0).view(-1, N)[s["slot"]]
        return {"Y": Y, "aux": _pack(bits)}
    return {"Y": Y, "aux": _unpad(s, Z, dt, T) if case["epilog"] == "GELU_AUX_BIAS" else None}


def run(s):
    if not own:
        return _plain(s)
    from gemm_epilogues_tcgen05_b200 import binding

    op = s["op"]
    if op == "mx_round":
        binding.gemm_epi_mx_quantize(s["X"], s["q"], s["scales"], transposed=s["case"]["transposed"])
        binding.gemm_epi_mx_dequantize(s["q"], s["scales"], s["values"])
        return s["values"]
    if op == "mx_linear":
        offsets = s["offsets"] if s["case"]["E"] else None
        binding.gemm_epi_mx_quantize(s["X"], s["Xq"], s["Xs"], offsets=offsets)
        s["plan"].gemm_epi_mx_execute(s["Xq"], s["Xs"], s["Wq"], s["Ws"], s["bias"], s["Y"], offsets=offsets)
        return s["Y"]
    if op == "wgrad":
        s["plan"].gemm_epi_grouped_wgrad_execute(s["X"], s["dZ"], s["offsets"], s["dW"], s["dbias"])
        return {"dW": s["dW"], "dbias": s["dbias"]}
    if op == "backward":
        s["plan"].gemm_epi_grouped_drelu_bgrad_execute(s["X"], s["W"], s["aux"], s["offsets"], s["dZ"], s["dbias"])
        return {"dZ": s["dZ"], "dbias": s["dbias"]}
    s["plan"].gemm_epi_grouped_execute(s["X"], s["W"], s["bias"], s["offsets"], s["Y"], s["aux"])
    return {"Y": s["Y"], "aux": s["aux"]}


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] == "mx_round":
        n = case["R"] * case["C"]
        return {"bytes": n * (2 + 4), "flops": 0}
    sizes = group_sizes(case)
    rows, active = int(sizes.sum()), int((sizes > 0).sum())
    K, N, o = case["K"], case["N"], 4 if case.get("out_f32") else 2
    flops = 2.0 * rows * K * N
    if case["op"] == "mx_linear":
        return {"bytes": rows * K * 2 + active * (N * K * (1 / 2 + 1 / 32) + N * 2) + rows * N * 2, "flops": flops}
    if case["op"] == "wgrad":
        return {"bytes": rows * (K + N) * 2 + case["E"] * (K * N * o + (K * 4 if case["dbias"] else 0)), "flops": flops}
    b = rows * K * 2 + active * K * N * 2 + rows * N * o
    if case["op"] == "backward":
        return {"bytes": b + rows * N / 8 + case["E"] * N * 4, "flops": flops}
    aux = {"RELU_AUX_BIAS": 1 / 8, "GELU_AUX_BIAS": 2}.get(case["epilog"], 0)
    return {"bytes": b + active * N * 2 + rows * N * aux, "flops": flops}


# --------------------------------------------------------------------- exact
def _exact_fp4(x):
    """Nearest representable value by distance, block by block, in 64 bits; of two at the same
    distance the one with the even code."""
    R, C = x.shape
    v = x.double().reshape(R * C // 32, 32)
    top = v.abs().max(dim=1, keepdim=True).values
    powers = torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device="cuda")
    # the largest power of two that is at most the block's largest magnitude, a quarter of it the scale
    at = torch.searchsorted(powers, top, right=True) - 1
    scale = torch.where(top > 0, powers[(at - 2).clamp(min=200 - 127)], powers[200 - 127])
    levels = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    out = torch.empty_like(v)
    for a in range(0, v.shape[0], 1 << 18):
        u = v[a:a + (1 << 18)] / scale[a:a + (1 << 18)]
        best, dist = torch.zeros_like(u), u.abs()
        for k in range(1, 8):
            d = (u.abs() - levels[k]).abs()
            better = (d < dist) | ((d == dist) & (k % 2 == 0))
            best, dist = torch.where(better, levels[k], best), torch.where(better, d, dist)
        out[a:a + (1 << 18)] = torch.copysign(best, u) * scale[a:a + (1 << 18)]
    return out.reshape(R, C)


def _exact_weight(q, scales, e, N, K):
    """Expert e's weight [N, K] in 64 bits, element by element from the stated layout."""
    n = torch.arange(N, device="cuda")[:, None]
    k = torch.arange(K, device="cuda")[None, :]
    byte = q[e].long()[n, k // 2]
    code = torch.where(k % 2 == 0, byte % 16, byte // 16)
    mag, ex = (code % 2).double(), (code // 2 % 4).double()
    powers = torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=torch.float64, device="cuda")
    val = torch.where(ex > 0, (1 + mag / 2) * powers[(ex - 1).long() + 127], mag / 2)
    b = k // 32
    tile = (e * ((N + 127) // 128) + n // 128) * ((K + 127) // 128) + b // 4
    at = tile * 512 + n % 32 * 16 + n % 128 // 32 * 4 + b % 4
    return torch.where(code >= 8, -val, val) * powers[scales[at].long()]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "mx_round":
        return _exact_fp4(s["X"].t().contiguous() if case["transposed"] else s["X"])
    T, K, N = case["T"], case["K"], case["N"]
    off = [0] + [int(v) for v in np.cumsum(s["sizes"])]
    spans = [(e, off[e], off[e + 1]) for e in range(len(s["sizes"]))]

    def act(z, epilog):
        if epilog.startswith("RELU"):
            return torch.clamp(z, min=0)
        if epilog.startswith("GELU"):
            return z * torch.special.ndtr(z)
        return z

    if op == "wgrad":
        dW = torch.zeros((case["E"], K, N), dtype=torch.float64, device="cuda")
        db = torch.zeros((case["E"], K), dtype=torch.float64, device="cuda")
        for e, a, b in spans:
            x = s["X"][a:b].double()
            dW[e] = x.t() @ s["dZ"][a:b].double()
            db[e] = x.sum(0)
        return {"dW": dW, "dbias": db if case["dbias"] else None}
    Y = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    if op == "mx_linear":
        X = _exact_fp4(s["X"])
        for e, a, b in spans:
            if b > a:
                z = X[a:b] @ _exact_weight(s["Wq"], s["Ws"], e, N, K).t()
                Y[a:b] = act(z + s["bias"][e].double() if case["epilog"] != "NONE" else z, case["epilog"])
        return Y
    Z = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    db = torch.zeros((max(case["E"], 1), N), dtype=torch.float64, device="cuda")
    col = torch.arange(N, device="cuda")
    for e, a, b in spans:
        w = s["W"][e].double()
        z = s["X"][a:b].double() @ (w.t() if case["w_nk"] else w)
        if op == "backward":
            on = (s["aux"][a:b][:, col // 32] >> (col % 32).to(torch.int32)) & 1
            Y[a:b] = z * on
            db[e] = Y[a:b].sum(0)
        else:
            Z[a:b] = z + s["bias"][e].double() if case["epilog"] != "NONE" else z
            Y[a:b] = act(Z[a:b], case["epilog"])
    if op == "backward":
        return {"dZ": Y, "dbias": db}
    if case["epilog"] == "RELU_AUX_BIAS":
        return {"Y": Y, "aux": None}
    return {"Y": Y, "aux": Z if case["epilog"] == "GELU_AUX_BIAS" else None}
