"""Cases of the gated feed-forward layer and of 4-bit weights with group scales.

Four operators:

* ``gated``     forward of a gated layer: both projections, the activation of
                the gate and the product with the up projection; for training
                also the pre-activations.
* ``dgated``    its backward: the gradient's product, then the gradients of
                both pre-activations, and their column sums where asked.
* ``w4_linear`` few rows times a weight held in 4 bits with a 16-bit scale
                (and, in half of the checkpoints, a zero point) for each group
                of 32, 64 or 128 columns; also as a gated layer.
* ``w4_round``  a weight to that form and back (what a conversion and its check
                run; what is held in 4 bits comes back as the values it stands
                for).

Operands of the 16-bit products lie on a fixed-point grid (7 bits and a sign),
as 8-bit checkpoints and activations give: every fp32 sum is then exact.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a small model's block: latency only
        dict(name="gated small decode", op="gated", dtype="bf16", T=1, K=1024, N=2048, act="SILU", w_nk=True, aux=False,
             bias=False, out_f32=False),
        # a batch of 8 tokens: the weight is streamed once
        dict(name="gated decode", op="gated", dtype="bf16", T=8, K=4096, N=11008, act="SILU", w_nk=False, aux=False,
             bias=False, out_f32=False),
        # odd sizes, biases, pre-activations kept, [out, in] checkpoints
        dict(name="gated ragged", op="gated", dtype="fp16", T=1003, K=1024, N=5000, act="GELU", w_nk=True, aux=True,
             bias=True, out_f32=False),
        # a training step
        dict(name="gated training", op="gated", dtype="bf16", T=4096, K=4096, N=11008, act="SILU", w_nk=False, aux=True,
             bias=False, out_f32=False),
        # backward of the odd sizes, with the biases' gradients
        dict(name="dgated ragged", op="dgated", dtype="fp16", T=1003, K=1024, N=5000, act="GELU", w_nk=True, bias=True,
             out_f32=False),
        # the training step's backward product
        dict(name="dgated training", op="dgated", dtype="bf16", T=4096, K=4096, N=11008, act="SILU", w_nk=False,
             bias=False, out_f32=False),
        # one token through a layer held in 4 bits
        dict(name="w4_linear one token", op="w4_linear", dtype="bf16", T=1, K=4096, N=11008, G=128, zeros=False,
             epilog="NONE", act="SILU"),
        # a few requests through a gated layer held in 4 bits with zero points
        dict(name="w4_linear gated", op="w4_linear", dtype="fp16", T=4, K=4096, N=11008, G=64, zeros=True,
             epilog="GATED", act="SILU"),
        # a serving batch of odd sizes, small groups
        dict(name="w4_linear batch", op="w4_linear", dtype="bf16", T=48, K=2080, N=5000, G=32, zeros=True,
             epilog="GELU_BIAS", act="SILU"),
        # a small layer's weight
        dict(name="w4_round small", op="w4_round", dtype="fp16", N=1000, K=1024, G=32, zeros=False),
        # a checkpoint's weight
        dict(name="w4_round weight", op="w4_round", dtype="bf16", N=11008, K=4096, G=128, zeros=True),
    ]


def draw(rng):
    def size(lo, hi, step):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(step, int(v / step) * step)

    op = rng.choice(["gated", "gated", "dgated", "dgated", "w4_linear", "w4_linear", "w4_linear", "w4_round"])
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("w4"):
        G = rng.choice([32, 64, 128])
        c = dict(op=op, dtype=dtype, N=size(8, 11008, 8), K=size(128, 11008, G), G=G, zeros=rng.random() < 0.5)
        if op == "w4_linear":
            c.update(T=size(1, 128, 1), epilog=rng.choice(["NONE", "BIAS", "RELU_BIAS", "GELU_BIAS", "GATED", "GATED"]),
                     act=rng.choice(["SILU", "GELU", "RELU"]))
        return c
    while True:
        T, K, N = size(1, 4096, 1), size(64, 8192, 8), size(64, 11008, 8)
        if T * K * N <= 4096 * 4096 * 11008 and K * N <= 4096 * 11008:
            break
    c = dict(op=op, dtype=dtype, T=T, K=K, N=N, act=rng.choice(["SILU", "SILU", "GELU", "RELU"]),
             w_nk=rng.random() < 0.5, bias=rng.random() < 0.4, out_f32=rng.random() < 0.2)
    if op == "gated":
        c.update(aux=rng.random() < 0.5)
    return c


# -------------------------------------------------------------------- inputs
def _grid(shape, unit, g, dtype):
    """Normal draws rounded to a grid of `unit`, std 32 units, at most 127."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(32).round_().clamp_(-127, 127).mul_(unit).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 23)
    op, dt, N, K = case["op"], DTYPES[case["dtype"]], case["N"], case["K"]
    s = {"case": case, "op": op, "dtype": dt}
    if op == "w4_round":
        G = case["G"]
        # rows of different size, few outliers
        w = torch.randn((N, K), generator=g, device="cuda") * torch.exp(
            0.5 * torch.randn((N, 1), generator=g, device="cuda")) / math.sqrt(K)
        s["W"] = torch.where(torch.rand((N, K), generator=g, device="cuda") < 1e-3, w * 8, w).to(dt)
        if own:
            from gemm_epilogues_tcgen05_b200 import binding

            s["q"], s["scales"], s["zeros"] = binding.w4_empty(N, K, dt, group=G, zeros=case["zeros"])
            s["values"] = torch.empty((N, K), dtype=torch.float32, device="cuda")
        return s
    T = case["T"]
    unit = 2.0 ** -(5 + round(math.log2(math.sqrt(K))))
    s["X"] = _grid((T, K), 2.0 ** -5, g, dt)
    if op == "w4_linear":
        G, gated = case["G"], case["epilog"] == "GATED"
        rows = 2 * N if gated else N
        # codes as a checkpoint has them: two a byte, the lower column in the low 4 bits
        s["codes"] = torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["s"] = ((torch.rand((rows, K // G), generator=g, device="cuda") + 0.5) / (5 * math.sqrt(K))).to(dt)
        s["z"] = (torch.randint(4, 12, (rows, K // G), generator=g, device="cuda", dtype=torch.uint8)
                  if case["zeros"] else None)
        s["bias"] = None if case["epilog"] in ("NONE", "GATED") else _grid((rows,), 2.0 ** -7, g, dt)
        if own:
            from gemm_epilogues_tcgen05_b200 import binding

            # the weight is laid out once, when a model is loaded
            shape = (2, N) if gated else (N,)
            s["w4"] = binding.w4_pack(s["codes"].view(*shape, -1), s["s"].view(*shape, -1),
                                      None if s["z"] is None else s["z"].view(*shape, -1))
            s["plan"] = binding.W4Plan(T, N, K, dt, case["epilog"], group=G, act=case["act"])
            s["Y"] = torch.zeros((T, N), dtype=dt, device="cuda")
        return s
    out = torch.float32 if case["out_f32"] else dt
    if op == "gated":
        s["W"] = _grid((2 * N, K) if case["w_nk"] else (K, 2 * N), unit, g, dt)
        s["bias"] = _grid((2 * N,), 2.0 ** -7, g, dt) if case["bias"] else None
    else:
        s["W2"] = _grid((N, K) if case["w_nk"] else (K, N), unit, g, dt)
        s["aux"] = torch.randn((T, 2 * N), generator=g, device="cuda").to(dt)
    if own:
        from gemm_epilogues_tcgen05_b200 import binding

        epi = "DGATED" if op == "dgated" else "GATED_AUX" if case["aux"] else "GATED"
        s["plan"] = binding.GatedPlan(T, N, K, dt, epi, act=case["act"], w_nk=case["w_nk"], out_f32=case["out_f32"])
        if op == "gated":
            s["H"] = torch.zeros((T, N), dtype=out, device="cuda")
            s["Z"] = torch.zeros((T, 2 * N), dtype=dt, device="cuda") if case["aux"] else None
        else:
            s["dZ"] = torch.zeros((T, 2 * N), dtype=out, device="cuda")
            s["dbias"] = torch.zeros((2 * N,), dtype=torch.float32, device="cuda") if case["bias"] else None
    return s


# --------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "SILU":
        return z / (1 + torch.exp(-z))
    if act == "GELU":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return torch.where(z > 0, z, torch.zeros((), device="cuda"))


def _dact(z, act):
    if act == "SILU":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "GELU":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return (z > 0).float()


def _w4_values(codes, s, z, G):
    """Codes, scales and zero points as a checkpoint has them -> the values, fp32."""
    q = torch.stack([codes & 15, codes >> 4], -1).view(s.shape[0], s.shape[1], G).float()
    q = q - (8.0 if z is None else z.float()[:, :, None])
    return (q * s.float()[:, :, None]).view(s.shape[0], -1)


def _w4_round(W, G, zeros):
    w = W.float().view(W.shape[0], -1, G)
    if zeros:
        lo, hi = w.amin(-1, keepdim=True).clamp(max=0), w.amax(-1, keepdim=True).clamp(min=0)
        s = ((hi - lo) / 15).to(W.dtype).float()
        z = (-lo / s).round().clamp(0, 15)
        q = ((w / s).round() + z).clamp(0, 15) - z
    else:
        s = (w.abs().amax(-1, keepdim=True) / 7).to(W.dtype).float()
        q = (w / s).round().clamp(-8, 7)
    return torch.where(s > 0, q * s, torch.zeros((), device="cuda")).view(W.shape)


def _plain(s):
    case, op, dt, N = s["case"], s["op"], s["dtype"], s["case"]["N"]
    if op == "w4_round":
        return _w4_round(s["W"], case["G"], case["zeros"])
    X = s["X"].float()
    if op == "w4_linear":
        Z = X @ _w4_values(s["codes"], s["s"], s["z"], case["G"]).t()
        if case["epilog"] == "GATED":
            return (_act(Z[:, :N], case["act"]) * Z[:, N:]).to(dt)
        if s["bias"] is not None:
            Z = Z + s["bias"].float()
        if case["epilog"] == "GELU_BIAS":
            Z = _act(Z, "GELU")
        return (_act(Z, "RELU") if case["epilog"] == "RELU_BIAS" else Z).to(dt)
    out = torch.float32 if case["out_f32"] else dt
    if op == "gated":
        W = s["W"].float()
        Z = X @ (W.t() if case["w_nk"] else W)
        if s["bias"] is not None:
            Z = Z + s["bias"].float()
        H = (_act(Z[:, :N], case["act"]) * Z[:, N:]).to(out)
        return {"H": H, "Z": Z.to(dt) if case["aux"] else None}
    W = s["W2"].float()
    dH = X @ (W.t() if case["w_nk"] else W)
    G, U = s["aux"][:, :N].float(), s["aux"][:, N:].float()
    dZ = torch.cat([dH * U * _dact(G, case["act"]), dH * _act(G, case["act"])], 1)
    return {"dZ": dZ.to(out), "dbias": dZ.sum(0) if case["bias"] else None}


def run(s):
    if not own:
        return _plain(s)
    from gemm_epilogues_tcgen05_b200 import binding

    op = s["op"]
    if op == "w4_round":
        G = s["case"]["G"]
        binding.gemm_epi_w4_quantize(s["W"], s["q"], s["scales"], s["zeros"], group=G)
        binding.gemm_epi_w4_dequantize(s["q"], s["scales"], s["zeros"], s["values"], group=G)
        return s["values"]
    if op == "w4_linear":
        s["plan"].gemm_epi_w4_execute(s["X"], *s["w4"], s["bias"], s["Y"])
        return s["Y"]
    if op == "gated":
        s["plan"].gemm_epi_gated_execute(s["X"], s["W"], s["bias"], s["H"], s["Z"])
        return {"H": s["H"], "Z": s["Z"]}
    s["plan"].gemm_epi_dgated_execute(s["X"], s["W2"], s["aux"], s["dZ"], s["dbias"])
    return {"dZ": s["dZ"], "dbias": s["dbias"]}


# ---------------------------------------------------------------------- work
def work(case):
    N, K, op = case["N"], case["K"], case["op"]
    if op == "w4_round":
        return {"bytes": N * K * (2 + 4), "flops": 0}
    T = case["T"]
    if op == "w4_linear":
        rows = 2 * N if case["epilog"] == "GATED" else N
        held = rows * K / 2 + rows * (K // case["G"]) * (3 if case["zeros"] else 2)
        bias = 0 if case["epilog"] in ("NONE", "GATED") else rows * 2
        return {"bytes": held + bias + T * (K + N) * 2, "flops": 2.0 * T * rows * K}
    o = 4 if case["out_f32"] else 2
    if op == "gated":
        return {"bytes": (T * K + 2 * N * K) * 2 + (4 * N if case["bias"] else 0) + T * N * o + (4 * T * N if case["aux"] else 0),
                "flops": 4.0 * T * N * K}
    return {"bytes": (T * K + N * K + 2 * T * N) * 2 + 2 * T * N * o + (8 * N if case["bias"] else 0),
            "flops": 2.0 * T * N * K}


# --------------------------------------------------------------------- exact
def _exact_act(z, act):
    """act(z) and its derivative in 64 bits."""
    if act == "SILU":
        p = torch.special.expit(z)
        return z * p, p + z * p * torch.special.expit(-z)
    if act == "GELU":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) * (1 / math.sqrt(2 * math.pi))
    return torch.clamp(z, min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))


def _exact_held(W, G, zeros):
    """Each group's nearest values, element by element, in 64 bits."""
    out = torch.empty(W.shape, dtype=torch.float64, device="cuda")
    for a in range(0, W.shape[1], G):
        w = W[:, a:a + G].double()
        lo, hi = w.min(1).values.clamp(max=0), w.max(1).values.clamp(min=0)
        top = torch.maximum(hi, -lo)
        s = ((hi - lo) / 15 if zeros else top / 7).to(W.dtype).double()[:, None]
        step = torch.where(s > 0, s, torch.ones_like(s))
        if zeros:
            z = torch.clamp(torch.round(-lo[:, None] / step), 0, 15)
            q = torch.clamp(torch.round(w / step) + z, 0, 15) - z
        else:
            q = torch.clamp(torch.round(w / step), -8, 7)
        out[:, a:a + G] = q * s
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, N, K = case["op"], case["N"], case["K"]
    if op == "w4_round":
        return _exact_held(s["W"], case["G"], case["zeros"])
    X = s["X"].double()
    if op == "w4_linear":
        k = torch.arange(K, device="cuda")
        code = (s["codes"].long()[:, k // 2] >> (4 * (k % 2))) % 16
        zero = s["z"].double()[:, k // case["G"]] if case["zeros"] else 8.0
        w = (code.double() - zero) * s["s"].double()[:, k // case["G"]]
        if case["epilog"] == "GATED":
            return _exact_act(X @ w[:N].t(), case["act"])[0] * (X @ w[N:].t())
        y = X @ w.t()
        if case["epilog"] != "NONE":
            y = y + s["bias"].double()
        return _exact_act(y, case["epilog"][:4])[0] if case["epilog"] in ("RELU_BIAS", "GELU_BIAS") else y
    if op == "gated":
        W = s["W"].double().t() if case["w_nk"] else s["W"].double()
        b = s["bias"].double() if case["bias"] else torch.zeros(2 * N, dtype=torch.float64, device="cuda")
        gate, up = X @ W[:, :N] + b[:N], X @ W[:, N:] + b[N:]
        return {"H": _exact_act(gate, case["act"])[0] * up, "Z": torch.cat([gate, up], 1) if case["aux"] else None}
    W = s["W2"].double().t() if case["w_nk"] else s["W2"].double()
    dH = X @ W
    a, d = _exact_act(s["aux"][:, :N].double(), case["act"])
    dG, dU = dH * s["aux"][:, N:].double() * d, dH * a
    return {"dZ": torch.cat([dG, dU], 1), "dbias": torch.cat([dG.sum(0), dU.sum(0)]) if case["bias"] else None}
