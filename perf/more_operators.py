"""The training side of a mixture-of-experts layer's feed-forward block, as cases to time and compare.

Three families: the gated block over groups of rows (both projections, silu(g) u, the product back), the
same with its backward pass from activations that were kept in 8 or 16 bits, and the weight gradient from
rows that are held in 8 bits.  Products are in 8-bit floating point with a power-of-two scale for each
block of 128, as everywhere in this repository; rows are pairs of a token and an expert, gathered from
the tokens.  Shapes follow the routing workloads: matrices of (4096, 2048) and (7168, 2048) next to smaller and odd
ones, top-8, and the pairs that one expert-parallel rank receives.

`run` computes a case in plain torch operations in 32 bits, or, where `own` is set, by the package's
entry points; `exact` gives the definition's values in 64 bits.
"""
import math

import numpy as np
import torch
import torch.nn.functional as F

own = False

BLOCK = 128


def listed():
    return [
        # decode of one token, top-8, through the grouped path: the weights' bytes count
        dict(name="block_step", kind="block", pairs=8, groups=8, hidden=4096, inter=2048, gather=8, masked=False),
        # a few sequences' tokens over many small groups
        dict(name="block_batch", kind="block", pairs=512, groups=16, hidden=2048, inter=1024, gather=8, masked=False),
        # prefill: a rank's share of 8192 tokens x top-8, rows gathered by pair
        dict(name="block_prefill", kind="block", pairs=65536, groups=8, hidden=4096, inter=2048, gather=8, masked=False),
        # prefill with skewed groups, an empty one and positions that no pair takes
        dict(name="block_ragged", kind="block", pairs=32749, groups=5, hidden=7168, inter=2048, gather=1, masked=True),
        # a small model's odd sizes, rows in order
        dict(name="block_odd", kind="block", pairs=5003, groups=3, hidden=1999, inter=1003, gather=0, masked=False),
        # fine-tuning on a short batch: a few rows in each group
        dict(name="train_small", kind="train", pairs=640, groups=8, hidden=4096, inter=1024, gather=8, masked=False,
             keep=8),
        # a rank's training microbatch with activations kept in 8 bits
        dict(name="train_rank", kind="train", pairs=65536, groups=8, hidden=4096, inter=2048, gather=8, masked=False,
             keep=8),
        # wide matrices, skewed groups, activations kept in 16 bits
        dict(name="train_wide", kind="train", pairs=16381, groups=3, hidden=7168, inter=2048, gather=1, masked=False,
             keep=16),
        # odd sizes with positions that no pair takes
        dict(name="train_odd", kind="train", pairs=3001, groups=5, hidden=1000, inter=777, gather=4, masked=True, keep=8),
        # gradient of the projections: the layer's 8-bit input gathered by pair, gradients in slot order
        dict(name="wgrad_rank", kind="wgrad", pairs=65536, groups=8, n=4096, k=4096, gather="x", div=8, masked=False),
        # gradient of the matrices back: the output's gradient gathered, 8-bit rows in slot order
        dict(name="wgrad_back", kind="wgrad", pairs=32749, groups=5, n=7168, k=2048, gather="dy", div=8, masked=True),
        # odd sizes, both in slot order
        dict(name="wgrad_odd", kind="wgrad", pairs=1201, groups=4, n=2001, k=999, gather="", div=1, masked=False),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even in its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    kind = rng.choice(("block", "block", "train", "train", "wgrad"))
    groups = rng.randint(1, 16)
    if kind == "wgrad":
        n, k = _spread(rng, 64, 7168), _spread(rng, 64, 4096)
        gather = rng.choice(("", "x", "dy"))
        return dict(kind=kind, pairs=min(_spread(rng, 1, 65536), int(8e11 / (n * k))), groups=groups, n=n, k=k,
                    gather=gather, div=rng.choice((1, 4, 8)) if gather else 1,
                    masked=bool(gather) and rng.random() < 0.4)
    hidden, inter, gather = _spread(rng, 64, 7168), _spread(rng, 64, 2048), rng.choice((0, 1, 4, 8))
    case = dict(kind=kind, pairs=min(_spread(rng, 1, 65536), int(4e11 / (hidden * inter))), groups=groups, hidden=hidden,
                inter=inter, gather=gather, masked=gather > 0 and rng.random() < 0.4)
    return dict(case, keep=rng.choice((8, 8, 16))) if kind == "train" else case


# ------------------------------------------------------------------------------------------------ inputs

def _padded(x, dim):
    """x with zeros up to a multiple of 128 along dim."""
    short = -x.shape[dim] % BLOCK
    return F.pad(x, [0, 0] * (x.dim() - 1 - dim % x.dim()) + [0, short]) if short else x


def _scale_code(amax):
    """The byte c of the smallest power of two 2**(c - 127) that brings amax to 448 at most."""
    bits = amax.float().view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(1, 254).to(torch.uint8)


def _power(code):
    """2**(code - 127) as float32."""
    return (code.to(torch.int32) << 23).view(torch.float32)


def _matrices(g, count, n, k):
    """Random matrices [count][n][k] in 8 bits: bytes [count][n][k up to 128], scale bytes for each 128 x 128."""
    w = _padded(_padded(torch.randn((count, n, k), generator=g, device="cuda") * k ** -0.5, 2), 1)
    t = w.view(count, w.shape[1] // BLOCK, BLOCK, w.shape[2] // BLOCK, BLOCK)
    code = _scale_code(t.abs().amax(dim=(2, 4)))
    q = (t * _power(254 - code)[:, :, None, :, None]).view(w.shape).to(torch.float8_e4m3fn)
    return q[:, :n].contiguous(), code.contiguous()


def _turned(q, code, cols):
    """The same matrices transposed: bytes [count][cols][n up to 128] and their scales."""
    t = _padded(q.view(torch.uint8)[:, :, :cols].transpose(1, 2), 2).contiguous()
    return t.view(torch.float8_e4m3fn), code.transpose(1, 2).contiguous()


def _sizes(seed, pairs, groups):
    """Skewed group sizes that sum to `pairs`; with three groups or more one is empty."""
    r = np.random.default_rng(int(seed) * 37 + 11)
    p = r.dirichlet(np.full(groups, 1.5))
    if groups > 2:
        p[int(r.integers(groups))] = 0
    return r.multinomial(pairs, p / p.sum())


def _activations(g, rows, cols):
    """Rows that differ in size, with a few large channels."""
    spread = torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    loud = 1 + 20 * (torch.rand(cols, generator=g, device="cuda") < 0.01).float()
    return torch.randn((rows, cols), generator=g, device="cuda") * spread * loud


def _rows_in_eight_bits(x):
    """[M][K] -> bytes [M][K up to 128] and scale bytes [M][blocks up to a multiple of 4], 127 past the blocks."""
    t = _padded(x, 1).view(x.shape[0], -1, BLOCK)
    code = _scale_code(t.abs().amax(dim=2))
    q = (t * _power(254 - code)[:, :, None]).view(x.shape[0], -1).to(torch.float8_e4m3fn)
    return q, F.pad(code, [0, -code.shape[1] % 4], value=127).contiguous()


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 17)
    s = dict(case=dict(case))
    pairs, groups = c["pairs"], c["groups"]
    sizes = _sizes(seed, pairs, groups)
    s["ends"] = [0] + [int(v) for v in np.cumsum(sizes)]
    s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")
    div = c["div"] if c["kind"] == "wgrad" else max(1, c["gather"])
    tokens = -(-pairs // div)
    s["rows"] = s["pos"] = None
    if c["gather"]:                                 # the pair at each position, and each pair's position
        order = torch.randperm(pairs, generator=g, device="cuda")
        pos = torch.empty_like(order)
        pos[order] = torch.arange(pairs, device="cuda")
        if c["masked"]:                             # positions that no pair takes
            free = torch.rand(pairs, generator=g, device="cuda") < 0.05
            pos[order[free]] = -1
            order[free] = -1
        s["rows"], s["pos"] = order.to(torch.int32), pos.to(torch.int32)
    if c["kind"] == "wgrad":
        s["dy"] = torch.randn((tokens if c["gather"] == "dy" else pairs, c["n"]), generator=g,
                              device="cuda").mul_(1e-3).to(torch.bfloat16)
        s["x"], s["x_scale"] = _rows_in_eight_bits(_activations(g, tokens if c["gather"] == "x" else pairs, c["k"]))
        return s
    s["x"] = _activations(g, tokens, c["hidden"]).to(torch.bfloat16)
    for name, n, k in (("gate", c["inter"], c["hidden"]), ("up", c["inter"], c["hidden"]),
                       ("down", c["hidden"], c["inter"])):
        s[name], s[name + "_scale"] = _matrices(g, groups, n, k)
    if c["kind"] == "train":
        # the matrices as the backward products take them; gate and up side by side, each up to whole blocks
        s["down_t"], s["down_t_scale"] = _turned(s["down"], s["down_scale"], c["inter"])
        (a, ac), (b, bc) = (_turned(s[name], s[name + "_scale"], c["hidden"]) for name in ("gate", "up"))
        s["both_t"] = torch.cat([a.view(torch.uint8), b.view(torch.uint8)], dim=2).view(torch.float8_e4m3fn)
        s["both_t_scale"] = torch.cat([ac, bc], dim=2)
        s["dout"] = torch.randn((tokens, c["hidden"]), generator=g, device="cuda").mul_(1e-3).to(torch.bfloat16)
        s["weights"] = torch.rand(pairs, generator=g, device="cuda")          # of the pairs, some nearly nothing
        s["weights"] *= torch.where(torch.rand(pairs, generator=g, device="cuda") < 0.02, 1e-6, 0.4)
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _rounded(x):
    """x with every 128 values of a row rounded to 8 bits, in float32."""
    t = _padded(x.float(), 1).view(x.shape[0], -1, BLOCK)
    code = _scale_code(t.abs().amax(dim=2, keepdim=True))
    q = (t * _power(254 - code)).to(torch.float8_e4m3fn).float() * _power(code)
    return q.view(x.shape[0], -1)[:, :x.shape[1]]


def _weights(q, code, k):
    """8-bit [..][N][K up to 128] with its block scales -> float32 [..][N][K]."""
    unit = _power(code).repeat_interleave(BLOCK, dim=-2)[..., :q.shape[-2], :].repeat_interleave(BLOCK, dim=-1)
    return (q.float() * unit)[..., :k]


def _gathered(x, rows, div):
    """x's row for each position; zeros where no pair is."""
    if rows is None:
        return x
    return x[rows.clamp(min=0).long() // div] * (rows >= 0).to(x.dtype)[:, None]


def _by_group(ends, rows, matrices):
    """Each group's rows times its matrix, transposed."""
    return torch.cat([rows[i:j] @ m.t() for i, j, m in zip(ends[:-1], ends[1:], matrices)])


def _plain_block(s):
    c, ends, rows, div = s["case"], s["ends"], s["rows"], max(1, s["case"]["gather"])
    gate, up = (_weights(s[name], s[name + "_scale"], c["hidden"]) for name in ("gate", "up"))
    down = _weights(s["down"], s["down_scale"], c["inter"])
    a = _gathered(_rounded(s["x"]), rows, div)
    g, u = _by_group(ends, a, gate), _by_group(ends, a, up)
    if c["kind"] == "block":
        return _by_group(ends, _rounded(F.silu(g) * u), down).to(torch.bfloat16)
    w = s["weights"] if rows is None else s["weights"][rows.clamp(min=0).long()]
    y = _by_group(ends, _rounded(F.silu(g) * u * w[:, None]), down).to(torch.bfloat16)
    g, u = (_rounded(g), _rounded(u)) if c["keep"] == 8 else (g.to(torch.bfloat16).float(), u.to(torch.bfloat16).float())
    d = _by_group(ends, _gathered(_rounded(s["dout"]), rows, div), down.transpose(1, 2))
    sig = torch.sigmoid(g)
    dots = (d * (g * sig * u)).sum(dim=1)
    d = d * w[:, None]
    dg, du = d * u * (sig * (1 + g * (1 - sig))), d * (g * sig)
    dx = _by_group(ends, _rounded(dg), gate.transpose(1, 2)) + _by_group(ends, _rounded(du), up.transpose(1, 2))
    if rows is not None:
        dots = torch.where(s["pos"] >= 0, dots[s["pos"].clamp(min=0).long()], 0.0)
    return dict(y=y, dx=dx.to(torch.bfloat16), inner=torch.cat([dg, du], dim=1).to(torch.bfloat16),
                weights=dots.to(torch.bfloat16))


def _plain_wgrad(s):
    c, rows = s["case"], s["rows"]
    kb = s["x"].shape[1] // BLOCK
    x = (s["x"].float() * _power(s["x_scale"][:, :kb]).repeat_interleave(BLOCK, dim=1))[:, :c["k"]]
    dy = s["dy"].float()
    if c["gather"]:
        gathered = _gathered(x if c["gather"] == "x" else dy, rows, c["div"])
        x, dy = (gathered, dy) if c["gather"] == "x" else (x, gathered)
    return torch.stack([dy[i:j].t() @ x[i:j] for i, j in zip(s["ends"][:-1], s["ends"][1:])])


# ------------------------------------------------------------------------------------------------ the package's calls

def _own(s):
    import moe_expert_load_layer_amd as ep
    c, rows = s["case"], s["rows"]
    if c["kind"] == "wgrad":
        return ep.ep_grouped_wgrad_mixed(s["dy"], s["x"], s["x_scale"], s["offsets"], cols=c["k"],
                                         dy_rows=rows if c["gather"] == "dy" else None,
                                         x_rows=rows if c["gather"] == "x" else None, rows_div=c["div"])
    div, train = max(1, c["gather"]), c["kind"] == "train"
    kinds = {8: torch.float8_e4m3fn, 16: torch.bfloat16}
    xq, xs = ep.ep_quant_rows(s["x"])
    h, hs, kept, ks = ep.ep_grouped_swiglu(
        xq, xs, s["gate"], s["gate_scale"], s["up"], s["up_scale"], s["offsets"], rows=rows, rows_div=div,
        weights=s["weights"] if train else None, keep=kinds[c["keep"]] if train else None)
    y = ep.ep_grouped_matmul(h, hs, s["down"], s["down_scale"], s["offsets"])
    if not train:
        return y
    dq, ds = ep.ep_quant_rows(s["dout"])
    inner, iq, iscale, weights = ep.ep_grouped_swiglu_backward(
        dq, ds, s["down_t"], s["down_t_scale"], kept, ks, s["offsets"], rows=rows, rows_div=div,
        weights=s["weights"], pos=s["pos"], weights_dtype=torch.bfloat16)
    dx = ep.ep_grouped_matmul(iq, iscale, s["both_t"], s["both_t_scale"], s["offsets"])
    return dict(y=y, dx=dx, inner=inner, weights=weights)


def run(state):
    if own:
        return _own(state)
    return _plain_wgrad(state) if state["case"]["kind"] == "wgrad" else _plain_block(state)


# ------------------------------------------------------------------------------------------------ work

def work(case):
    c, m = case, case["pairs"]
    used = max(1, c["groups"] - (c["groups"] > 2)) if m >= 4 * c["groups"] else min(m, c["groups"])
    if c["kind"] == "wgrad":
        t = -(-m // c["div"])
        return dict(bytes=2 * c["n"] * (t if c["gather"] == "dy" else m) + c["k"] * (t if c["gather"] == "x" else m) +
                    4 * c["groups"] * c["n"] * c["k"] + (4 * m if c["gather"] else 0), flops=2 * m * c["n"] * c["k"])
    h, i, t = c["hidden"], c["inter"], -(-m // max(1, c["gather"]))
    # each matrix once (the backward products read theirs again), the tokens' rows, the pairs' rows
    forward = 3 * used * h * i + 2 * t * h + 2 * m * h
    if c["kind"] == "block":
        return dict(bytes=forward, flops=6 * m * h * i)
    return dict(bytes=forward + 3 * used * h * i + 2 * t * h + 2 * m * h + 4 * m * i + 10 * m, flops=12 * m * h * i)


# ------------------------------------------------------------------------------------------------ 64 bits

def _pow2(e):
    """2**e in float64, exactly, for whole numbers e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _held(x):
    """Float64 rows as 8 bits hold them: blocks of 128 scaled to 448 at most, 4 bits of mantissa, ties to even."""
    out = torch.empty_like(x)
    for at in range(0, x.shape[1], 128):
        t = x[:, at:at + 128]
        mant, ex = torch.frexp(t.abs().amax(dim=1, keepdim=True))
        unit = _pow2((ex + (mant > 0.875).int() - 9).clamp(min=-126))
        v = t / unit
        step = _pow2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 4)
        out[:, at:at + 128] = torch.round(v / step) * step * unit
    return out


def _scaled(q, code, k):
    """One matrix [N][K up to 128] with a scale for each 128 x 128 -> float64 [N][K]."""
    unit = _pow2(code.int() - 127)
    n, cols = (torch.arange(size, device=q.device) // 128 for size in q.shape)
    return (q.double() * unit[n][:, cols])[:, :k]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    m, ends = c["pairs"], s["ends"]
    pair = torch.arange(m, device="cuda") if s["rows"] is None else s["rows"].long()
    if c["kind"] == "wgrad":
        out = torch.zeros((c["groups"], c["n"], c["k"]), dtype=torch.float64, device="cuda")
        unit = _pow2(s["x_scale"].int() - 127)[:, torch.arange(c["k"], device="cuda") // 128]
        x, dy = s["x"][:, :c["k"]].double() * unit, s["dy"].double()
        for e in range(c["groups"]):
            at = torch.arange(ends[e], ends[e + 1], device="cuda")
            at = at[pair[at] >= 0]
            of = pair[at] // c["div"]
            out[e] = dy[of if c["gather"] == "dy" else at].t() @ x[of if c["gather"] == "x" else at]
        return out
    h, i, train, div = c["hidden"], c["inter"], c["kind"] == "train", max(1, c["gather"])
    f64 = dict(dtype=torch.float64, device="cuda")
    y, x = torch.zeros((m, h), **f64), _held(s["x"].double())
    if train:
        dout = _held(s["dout"].double())
        dx, inner, weights = torch.zeros((m, h), **f64), torch.zeros((m, 2 * i), **f64), torch.zeros(m, **f64)
    for e in range(c["groups"]):
        at = torch.arange(ends[e], ends[e + 1], device="cuda")
        at = at[pair[at] >= 0]
        if not len(at):
            continue
        p, t = pair[at], pair[at] // div
        gate, up = (_scaled(s[name][e], s[name + "_scale"][e], h) for name in ("gate", "up"))
        down = _scaled(s["down"][e], s["down_scale"][e], i)
        g, u = x[t] @ gate.t(), x[t] @ up.t()
        w = s["weights"][p].double()[:, None] if train else 1.0
        y[at] = _held(g / (1 + torch.exp(-g)) * u * w) @ down.t()
        if not train:
            continue
        g, u = (_held(g), _held(u)) if c["keep"] == 8 else (g.to(torch.bfloat16).double(), u.to(torch.bfloat16).double())
        d = dout[t] @ down
        sig = 1 / (1 + torch.exp(-g))
        weights[p] = (d * u * g * sig).sum(dim=1)
        dg = w * d * u * sig * (1 + g - g * sig)
        du = w * d * g * sig
        dx[at] = _held(dg) @ gate + _held(du) @ up
        inner[at] = torch.cat([dg, du], dim=1)
    return dict(y=y, dx=dx, inner=inner, weights=weights) if train else y
