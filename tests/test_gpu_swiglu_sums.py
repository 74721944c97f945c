"""The precision of the gated block's sums, which are rounded to 8 bits at once: fp32's for every number of rows,
columns and terms.

Whole numbers: every partial sum is a multiple of 2^-9 below 2^14, so fp32's sums are exact in any order.  One product
of 448 in 8 next to others below 2^-13 of it, which cancels against the next 8's, is what the 8-bit instruction cannot
add: it drops all but the large one.

Random values: each of K additions is off by 2^-24 of a partial sum.  With signs at random the partial sums are about
R = sqrt(sum (x w)^2), and the errors add like a random walk: sqrt(K) 2^-24 R.  16 times that covers partial sums of
4 R and four standard deviations.  With a channel in fifty 20 times larger the 8-bit instruction is off by about 1.5e-4 R,
16 sqrt(1000) 2^-24 is 3e-5."""
import numpy as np
import pytest
import torch

import swiglu_ref as S
from test_gpu_swiglu import BF16, FP8, Case, _split

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


# sizes of groups, hidden, inter: tiles of 64, 128 and 256 rows, few and many values, columns and terms
SHAPES = [([3, 9], 512, 129), ([300, 211], 640, 300), ([60] * 40, 704, 1300), ([1000, 2001, 0], 1000, 777),
          ([2100, 1903], 520, 2020), ([9000, 8001], 400, 1100), ([5000, 4000], 1024, 200)]


def _name(v):
    return f"{sum(v)}in{len(v)}" if isinstance(v, list) else str(v)


def _whole(rng, rows, cols, size):
    """Whole numbers below `size` but for every eighth, and the eighths' places."""
    a = rng.integers(-size, size + 1, (rows, cols)).astype(np.float64)
    return a, np.arange(0, cols - cols % 16, 8)


def _loud_rows(rng, M, K):
    """Multiples of 2^-9 below 2^-6, and 448."""
    a, loud = _whole(rng, M, K, 7)
    a *= 2.0 ** -9
    a[:, loud] = 448
    return torch.from_numpy(a.astype(np.float32))


def _turns(rng, G, N, K):
    """Whole numbers up to 3, and 1 and -1 in turn where the rows are loud."""
    a, loud = _whole(rng, G * N, K, 3)
    a[:, loud] = 1 - 2 * (loud // 8 % 2)
    return torch.from_numpy(a.reshape(G, N, K).astype(np.float32))


class Whole:
    def __init__(self, dev, sizes, hidden, inter):
        rng = np.random.default_rng(hidden + inter)
        self.sizes, self.M, G = sizes, sum(sizes), len(sizes)
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=dev)
        self.x = _loud_rows(rng, self.M, hidden).to(dev)
        self.a, self.b = (_turns(rng, G, inter, hidden).to(dev) for _ in range(2))
        self.xq = ep.ep_quant_rows(self.x)
        self.aq, self.bq = ep.ep_quant_blocks(self.a), ep.ep_quant_blocks(self.b)
        assert torch.equal(S.values(*self.xq)[:, :hidden], self.x.double())
        for g in range(G):
            assert torch.equal(S.matrix(self.aq[0][g], self.aq[1][g], hidden), self.a[g].double())

    def product(self, w):
        ends = np.concatenate([[0], np.cumsum(self.sizes)])
        return torch.cat([self.x[i:j].double() @ w[g].double().t() for g, (i, j) in enumerate(zip(ends[:-1], ends[1:]))])


@pytest.mark.parametrize("sizes,hidden,inter", SHAPES, ids=_name)
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_whole_numbers_forward(dev, sizes, hidden, inter, keep):
    c = Whole(dev, sizes, hidden, inter)
    g, u = c.product(c.a), c.product(c.b)
    assert float(g.abs().max()) < 8 and float(g.abs().min(dim=1).values.max()) < 1 < float(g.abs().max())
    h, hs, kept, ks = ep.ep_grouped_swiglu(*c.xq, *c.aq, *c.bq, c.offsets, keep=keep)
    if keep is BF16:
        assert torch.equal(kept, torch.cat([g, u], 1).float().to(BF16))
    else:
        wide, n = -(-inter // 128) * 128, -(-inter // 128)
        for want, at in ((g, 0), (u, 1)):
            scale = torch.full((c.M, -(-n // 4) * 4), 127, dtype=torch.uint8, device=dev)
            scale[:, :n] = ks[:, at * n:(at + 1) * n]
            S.check_fp8(kept[:, at * wide:(at + 1) * wide], scale, want, torch.zeros_like(want), "gu"[at])
    s = torch.sigmoid(g)
    want = g * s * u
    S.check_fp8(h, hs, want, want.abs() * (S.HARDWARE + 2.0 ** -22) + (g * u).abs() * S.TINY, "h")


def _sum_bound(x, w):
    return 16 * x.shape[1] ** 0.5 * 2.0 ** -24 * (x.square() @ w.square().t()).sqrt()


def _loud(dev, sizes, hidden, inter, div):
    """A case with one token a hundred times larger than the others."""
    c = Case(dev, sizes, hidden, inter, div, masked=div > 0, extra=3)
    c.x[5 % c.tokens] *= 128
    c.dy[7 % c.tokens] *= 128
    c.xq, c.dq = ep.ep_quant_rows(c.x), ep.ep_quant_rows(c.dy)
    return c


@pytest.mark.parametrize("sizes,hidden,inter", SHAPES, ids=_name)
@pytest.mark.parametrize("div", [0, 4])
def test_random_forward(dev, sizes, hidden, inter, div):
    c = _loud(dev, sizes, hidden, inter, div)
    x = S.values(*c.xq)[:, :hidden]
    names = ("g", "eg", "u", "eu", "h", "eh")
    for out, e, at, t, w in c._per_group(names, inter):
        if e is None:
            r = out
            break
        gate, up = (S.matrix(q[e], s[e], hidden) for q, s in (c.gate, c.up))
        g, _, u, _, h, _ = S.forward(x[t], gate, up, w)
        eg, eu = _sum_bound(x[t], gate), _sum_bound(x[t], up)
        a = g * torch.sigmoid(g)
        ea = 1.1 * eg + a.abs() * S.HARDWARE + g.abs() * S.TINY
        eh = w.abs() * (ea * u.abs() + a.abs() * eu + ea * eu) + h.abs() * 2.0 ** -22
        for name, v in zip(names, (g, eg, u, eu, h, eh)):
            out[name][at] = v
    h, hs, kept, ks = c.run_forward(FP8)
    S.check_fp8(h, hs, r["h"], r["eh"], "h")
    wide, n = -(-inter // 128) * 128, -(-inter // 128)
    for name, at in (("g", 0), ("u", 1)):
        scale = torch.full((c.M, -(-n // 4) * 4), 127, dtype=torch.uint8, device=dev)
        scale[:, :n] = ks[:, at * n:(at + 1) * n]
        S.check_fp8(kept[:, at * wide:(at + 1) * wide], scale, r[name], r["e" + name], name)
    for name, got in zip(("g", "u"), _split(c.run_forward(BF16)[2], inter, inter)):
        S.check_bf16(got, r[name], r["e" + name], name)


def _bytes(*tensors):
    return [t.view(torch.uint8) for t in tensors if t is not None]


@pytest.mark.parametrize("sizes,hidden,inter", [([2100, 1903], 520, 2020), ([700, 0, 801], 1000, 777),
                                                ([9000, 8001], 400, 300)], ids=_name)
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_a_row_does_not_depend_on_the_others(dev, sizes, hidden, inter, keep):
    """A few rows of each group by themselves: the same bytes as among all of them."""
    c = Case(dev, sizes, hidden, inter, 4, True)
    h, hs, kept, ks = c.run_forward(keep)
    starts = np.concatenate([[0], np.cumsum(sizes)])[:-1]
    for count in (1, 33, 140):
        taken = [np.arange(s + n // 3, min(s + n, s + n // 3 + count)) for s, n in zip(starts, sizes)]
        at = torch.from_numpy(np.concatenate(taken)).to(dev)
        off = torch.tensor(np.concatenate([[0], np.cumsum([len(t) for t in taken])]), dtype=torch.int32, device=dev)
        rows = c.rows[at]
        h1, hs1, kept1, ks1 = ep.ep_grouped_swiglu(*c.xq, *c.gate, *c.up, off, rows=rows, rows_div=4, weights=c.weights,
                                                   keep=keep)
        assert all(torch.equal(a, b) for a, b in zip(
            _bytes(h1, hs1, kept1, ks1), _bytes(h.view(torch.uint8)[at], hs[at], kept.view(torch.uint8)[at],
                                                None if ks is None else ks[at]))), count


def _held(v):
    """Float64 rows as 8 bits hold them."""
    t = S.blocks(v)
    unit = torch.exp2(S.scale_code(t.abs().amax(2)) - 127)[:, :, None]
    return (S.round_fp8(t / unit) * unit).flatten(1)[:, :v.shape[1]]


@pytest.mark.parametrize("sizes,hidden,inter", SHAPES[3:], ids=_name)
def test_outputs_are_off_by_little_more_than_their_rounding(dev, sizes, hidden, inter):
    """The product of h, in norm, against its definition in 64 bits.

    A sum off by 2^-18 of a value passes a border of the 8 bits (steps of 2^-4 at most) once in 2^13 values; the output
    is off by 2^-6.5 2^-4 = 7e-4 then, beside 1.7e-3 of its own rounding to bf16: 1.1 times that, and 1.5 are granted, as
    rows are not of one size.  (Sums off by 2^-14 would make it 3e-3.)"""
    c = Case(dev, sizes, hidden, inter, 4, True)
    rng = np.random.default_rng(1)
    G = len(sizes)
    draw = lambda n, k: torch.from_numpy((rng.normal(0, 1, (G, n, k)) / np.sqrt(k)).astype(np.float32)).to(dev)  # noqa: E731
    down = ep.ep_quant_blocks(draw(hidden, inter))
    x = S.values(*c.xq)[:, :hidden]
    y = torch.zeros((c.M, hidden), dtype=torch.float64, device=dev)
    h, hs, _, _ = c.run_forward(None)
    for _, e, at, t, w in c._per_group((), 0):
        if e is None:
            break
        g, u = (x[t] @ S.matrix(v[e], s[e], hidden).t() for v, s in (c.gate, c.up))
        y[at] = _held(w * g * torch.sigmoid(g) * u) @ S.matrix(down[0][e], down[1][e], inter).t()
    got = ep.ep_grouped_matmul(h, hs, *down, c.offsets)
    own = float((y.float().to(BF16).double() - y).norm())
    assert float((got.double() - y).norm()) <= 1.5 * own


@pytest.mark.parametrize("sizes,hidden,inter", SHAPES, ids=_name)
def test_sums_of_8_bits_where_asked(dev, sizes, hidden, inter):
    """sums8: what is kept in bf16 has ep_grouped_matmul's sums, bit for bit, and h lies within their bound."""
    c = Case(dev, sizes, hidden, inter, 4, True, 3)
    h, hs, kept, _ = c.run_forward(BF16, sums8=True)
    r = c.forward()
    S.check_fp8(h, hs, r["h"], r["eh"], "h")
    for (w, scale), got in zip((c.gate, c.up), _split(kept, inter, inter)):
        apart = ep.ep_grouped_matmul(*c.xq, w, scale, c.offsets, rows=c.rows, rows_div=4)
        assert torch.equal(got, apart)
    eight = c.run_forward(FP8, sums8=True)
    assert all(torch.equal(a, b) for a, b in zip(_bytes(*eight[:2]), _bytes(h, hs)))
    # alone as among the others
    at = c.total // 3
    e = int(np.searchsorted(np.cumsum(sizes), at, side="right"))
    off = torch.tensor([0] * (e + 1) + [1] * (len(sizes) - e), dtype=torch.int32, device=dev)
    h1, hs1, kept1, _ = ep.ep_grouped_swiglu(*c.xq, *c.gate, *c.up, off, rows=c.rows[at:at + 1], rows_div=4,
                                             weights=c.weights, keep=BF16, sums8=True)
    assert all(torch.equal(a[0], b[at]) for a, b in zip(_bytes(h1, hs1, kept1), _bytes(h, hs, kept)))
