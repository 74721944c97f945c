"""The gated block over groups, forward and backward, in float64 on the tensors' device, with the bounds of what
the kernels may differ by.  Definitions only, no code of the package.

Products in 8 bits: 7 2^-13 sum |x w| (7 dropped rests below 2^-13 of the largest of each 8 products).  The sigmoid
through the hardware's exponential and reciprocal: the exponent is off by 2^-24 |g| log2 e, the two steps by an ulp
each, together below 2^-16 of a value for |g| <= 128; and it gives 0 for results below the least normal float, 2^-126,
which sigmoid(g) is from g = -87.4 on: there it is off by all of itself, less than 2^-126 (TINY).  What is rounded afterwards is checked by the rounding's
monotony: the output lies between the roundings of value - bound and value + bound."""
import torch

DROPPED = 7 * 2.0 ** -13
HARDWARE = 2.0 ** -16
TINY = 2.0 ** -126


def _levels(device):
    bits = torch.arange(0x7F, device=device)
    e, m = bits >> 3, (bits & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))


def round_fp8(v):
    """To the nearest e4m3 value, ties to even; |v| above 448 becomes 448."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    q = torch.round(a / step) * step
    assert torch.isin(q, _levels(v.device)).all()
    return torch.copysign(q, v)


def scale_code(amax):
    c = torch.ceil(torch.log2((amax / 448.0).clamp(min=2.0 ** -140)))
    c = torch.where(448.0 * torch.exp2(c - 1) >= amax, c - 1, torch.where(448.0 * torch.exp2(c) < amax, c + 1, c))
    return (c + 127).clamp(1, 254)


def blocks(x):
    """[M][N] -> [M][blocks][128], zeros past N."""
    return torch.nn.functional.pad(x, [0, -x.shape[1] % 128]).view(x.shape[0], -1, 128)


def values(q, scale):
    """Bytes and scale bytes [M][>= blocks] -> float64 [M][blocks * 128]."""
    kb = q.shape[1] // 128
    unit = torch.exp2(scale[:, :kb].double() - 127)
    return q.double() * unit.repeat_interleave(128, dim=1)


def matrix(q, scale, cols):
    """One matrix in 8 bits -> float64."""
    unit = torch.exp2(scale.double() - 127).repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)
    return (q.double() * unit)[:, :cols]


def check_fp8(q, scale, want, bound, what):
    """q, scale: rows in 8 bits of `want` known to `bound`."""
    w, e = blocks(want), blocks(bound)
    kb = w.shape[1]
    assert q.shape == (want.shape[0], kb * 128), what
    assert (scale[:, kb:] == 127).all() and scale.shape[1] == -(-kb // 4) * 4, what
    low, high = scale_code((w.abs() - e).clamp(min=0).amax(2)), scale_code((w.abs() + e).amax(2))
    code = scale[:, :kb].double()
    assert ((low <= code) & (code <= high)).all(), f"{what}: scales"
    unit = torch.exp2(code - 127)[:, :, None]
    got = blocks(q.double()) * unit
    below, above = round_fp8((w - e) / unit) * unit, round_fp8((w + e) / unit) * unit
    # a value that the smaller of two scales cannot hold is not there
    assert ((below <= got) & (got <= above)).all(), f"{what}: {int((~((below <= got) & (got <= above))).sum())} values"
    assert (blocks(q.double()).view(want.shape[0], -1)[:, want.shape[1]:] == 0).all(), f"{what}: past the columns"


def check_bf16(got, want, bound, what):
    """got: bf16 of `want` known to `bound`; float32's own rounding on the way to bf16 is a 2^-24 more."""
    e = bound + want.abs() * 2.0 ** -22
    low, high = ((want + s * e).float().to(torch.bfloat16).double() for s in (-1, 1))
    # two roundings (to float32 and to bf16) may pass a border by 2^-24
    fine = (low - want.abs() * 2.0 ** -22 <= got.double()) & (got.double() <= high + want.abs() * 2.0 ** -22)
    assert fine.all(), f"{what}: {int((~fine).sum())} of {fine.numel()}"


def forward(x, gate, up, weights):
    """One group's rows: float64 g, u, h and their bounds."""
    g, u = x @ gate.t(), x @ up.t()
    eg, eu = DROPPED * (x.abs() @ gate.abs().t()), DROPPED * (x.abs() @ up.abs().t())
    s = torch.sigmoid(g)
    a = g * s
    h = a * u * weights
    ea = 1.1 * eg + a.abs() * HARDWARE + g.abs() * TINY    # |silu'| < 1.1
    eh = weights.abs() * (ea * u.abs() + a.abs() * eu + ea * eu) + h.abs() * 2.0 ** -22
    return g, eg, u, eu, h, eh


def backward(d, ed, g, u, weights):
    """Rows of d known to ed -> dg, du, the terms of dw, each with its bound."""
    s = torch.sigmoid(g)
    slope, a = s * (1 + g * (1 - s)), g * s
    es = HARDWARE * s + TINY
    eslope = 2 * es * (1 + g.abs())            # of s, in both of its places
    dg, du, dw = weights * d * u * slope, weights * d * a, d * a * u
    edg = (weights * u).abs() * (slope.abs() * ed + (d.abs() + ed) * eslope) + dg.abs() * 2.0 ** -21
    ea = g.abs() * es
    edu = weights.abs() * (a.abs() * ed + (d.abs() + ed) * ea) + du.abs() * 2.0 ** -21
    edw = u.abs() * (a.abs() * ed + (d.abs() + ed) * ea) + dw.abs() * 2.0 ** -21
    return dg, edg, du, edu, dw, edw
