"""Codes of 4-bit weights where a quotient decides a rounding: every 16-bit value of a group's range against
the definition in 64 bits, with zero points, with odd scales, and at both ends of bf16's exponents."""
import pytest
import torch

from gemm_epilogues_tcgen05_b200 import gemm_epi_w4_dequantize, w4_quantize

from test_w4_gpu import DT, reference_codes, unpack, values

pytestmark = pytest.mark.gpu


def check(W, G, zeros):
    q, s, z = w4_quantize(W, group=G, zeros=zeros)
    codes, sc, ze = unpack(q, s, z, *W.shape, G)
    rc, rs, rz = reference_codes(W, G, zeros)
    assert torch.equal(sc, rs)
    assert not zeros or torch.equal(ze, rz)
    assert torch.equal(codes, rc)
    out = torch.empty(W.shape, dtype=torch.float32, device="cuda")
    gemm_epi_w4_dequantize(q, s, z, out, group=G)
    assert torch.equal(out.double(), values(rc, rs, rz if zeros else None, G))
    return rs


def groups(v, ends):
    """Rows of 32: 30 values of v and the group's ends."""
    v = torch.cat([v, v.new_zeros((-len(v)) % 30)]).view(-1, 30)
    return torch.cat([v, torch.tensor([ends], device="cuda").to(v.dtype).expand(len(v), 2)], 1).contiguous()


def finite(dt):
    bits = torch.arange(-32768, 32768, device="cuda", dtype=torch.int32).to(torch.int16).view(dt)
    return bits[bits.isfinite()]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [False, True])
def test_odd_scales(dt, zeros):
    """Scales of every seventh mantissa (fp16: every 91st), odd ones among them, each with all values of its range:
    quotients that are ties, and those next to one."""
    dt = DT[dt]
    v, bits = finite(dt), 8 if dt is torch.bfloat16 else 11
    seen = 0
    for m in range(2 ** (bits - 1), 2 ** bits, 7 if bits == 8 else 91):
        s = m * 2.0 ** -(bits + 3)
        lo, hi = (-7.0 * s, 8.0 * s) if zeros else (-7.0 * s, 7.0 * s)
        for shift in ((0.0, 3.5) if zeros else (0.0,)):  # (another zero point)
            a, b = lo + shift * s, hi + shift * s
            ends = torch.tensor([a, b], device="cuda").to(dt)
            in_range = v[(v >= ends[0]) & (v <= ends[1])]
            tiny = in_range.abs().double() < s / 64     # thousands of values that are 0
            rs = check(groups(torch.cat([in_range[~tiny], in_range[tiny][::97]]), [a, b]), 32, zeros)
            seen += rs.unique().numel()
    assert seen >= 12


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** -100, 0.9e-30, 1.0e-30, 1.1e-30, 1.5 * 2.0 ** -126, 2.0 ** -126, 2.0 ** -128, 3 * 2.0 ** -133, 2.0 ** -133,
                                   2.0 ** 100, 2.0 ** 123, 1.9 * 2.0 ** 123])
def test_ends_of_bf16(scale, zeros):
    """Around 1e-30, where the quotient's form changes, below the normal numbers, and near the largest."""
    v = finite(torch.bfloat16)
    ends = [-7 * scale, (8 if zeros else 7) * scale]
    ends = torch.tensor(ends, device="cuda", dtype=torch.float64).to(torch.bfloat16)
    in_range = v[(v >= ends[0]) & (v <= ends[1])]
    keep = in_range.double().abs() >= scale / 32
    check(groups(torch.cat([in_range[keep], in_range[~keep][::211]]), ends.tolist()), 32, zeros)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_random_groups_of_few_bits(dt, zeros, G):
    """Weights that are small multiples of their group's unit, the scale twice the unit: half of the quotients are ties."""
    g = torch.Generator(device="cuda")
    g.manual_seed(G)
    W = torch.randint(-14, 15, (512, 1024), generator=g, device="cuda").double()
    unit = 2.0 ** torch.randint(-14, 4, (512, 1024 // G, 1), generator=g, device="cuda").double()
    W = (W.view(512, -1, G) * unit).view(512, 1024)
    W.view(512, -1, G)[..., 0] = -14 * unit[..., 0]
    W.view(512, -1, G)[..., 1] = (16 if zeros else 14) * unit[..., 0]
    check(W.to(DT[dt]), G, zeros)
