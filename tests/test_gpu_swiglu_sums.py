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


@pytest.mark.parametrize("sizes,hidden,inter", SHAPES, ids=_name)
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_whole_numbers_backward(dev, sizes, hidden, inter, keep):
    c = Whole(dev, sizes, hidden, inter)
    d = c.product(c.a)
    rng = np.random.default_rng(3)
    both = torch.from_numpy(rng.normal(0, 1, (c.M, 2 * inter)).astype(np.float32)).to(BF16).to(dev)
    wide, n = -(-inter // 128) * 128, -(-inter // 128)
    kept, ks, full = both, None, both.double()
    if keep is FP8:
        apart = torch.zeros((c.M, 2 * wide), dtype=BF16, device=dev)
        for at in range(2):
            apart[:, at * wide:at * wide + inter] = both[:, at * inter:(at + 1) * inter]
        kept, ks = ep.ep_quant_rows(apart)
        full = S.values(kept, ks)
    w = torch.from_numpy(rng.random(c.M).astype(np.float32)).to(dev)
    grad, q, qs, dw = ep.ep_grouped_swiglu_backward(*c.xq, *c.aq, kept, ks, c.offsets, weights=w)
    kg, ku = _split(full, inter, wide if keep is FP8 else inter)
    dg, edg, du, edu, terms, et = S.backward(d, torch.zeros_like(d), kg, ku, w.double()[:, None])
    for name, got, at, want, e in zip(("dg", "du"), _split(grad, inter, inter), (0, 1), (dg, du), (edg, edu)):
        S.check_bf16(got, want, e, name)
        scale = torch.full((c.M, -(-n // 4) * 4), 127, dtype=torch.uint8, device=dev)
        scale[:, :n] = qs[:, at * n:(at + 1) * n]
        S.check_fp8(q[:, at * wide:(at + 1) * wide], scale, want, e, name + " in 8 bits")
    assert ((dw.double() - terms.sum(1)).abs() <= et.sum(1) + (128 + n) * 2.0 ** -24 * terms.abs().sum(1)).all()


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


@pytest.mark.parametrize("sizes,hidden,inter", SHAPES, ids=_name)
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_random_backward(dev, sizes, hidden, inter, keep):
    c = _loud(dev, sizes, hidden, inter, 4)
    _, _, kept, ks = c.run_forward(keep)
    wide, n = -(-inter // 128) * 128, -(-inter // 128)
    kg, ku = _split(S.values(kept, ks) if keep is FP8 else kept.double(), inter, wide if keep is FP8 else inter)
    dy = S.values(*c.dq)[:, :hidden]
    names = ("dg", "edg", "du", "edu", "dw", "edw")
    for out, e, at, t, w in c._per_group(names, inter):
        if e is None:
            r = out
            break
        down = S.matrix(c.down_t[0][e], c.down_t[1][e], hidden)
        for name, v in zip(names, S.backward(dy[t] @ down.t(), _sum_bound(dy[t], down), kg[at], ku[at], w)):
            out[name][at] = v
    grad, q, qs, dw = c.run_backward(kept, ks)
    for name, got, at in zip(("dg", "du"), _split(grad, inter, inter), (0, 1)):
        S.check_bf16(got, r[name], r["e" + name], name)
        scale = torch.full((c.M, -(-n // 4) * 4), 127, dtype=torch.uint8, device=dev)
        scale[:, :n] = qs[:, at * n:(at + 1) * n]
        S.check_fp8(q[:, at * wide:(at + 1) * wide], scale, r[name], r["e" + name], name + " in 8 bits")
    at = c.pos.long()
    want, e = (torch.where(at >= 0, v[at.clamp(min=0)], 0.0)
               for v in (r["dw"].sum(1), r["edw"].sum(1) + (128 + n) * 2.0 ** -24 * r["dw"].abs().sum(1)))
    assert ((dw.double() - want).abs() <= e).all()


def _bytes(*tensors):
    return [t.view(torch.uint8) for t in tensors if t is not None]


@pytest.mark.parametrize("sizes,hidden,inter", [([2100, 1903], 520, 2020), ([700, 0, 801], 1000, 777),
                                                ([9000, 8001], 400, 300)], ids=_name)
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_a_row_does_not_depend_on_the_others(dev, sizes, hidden, inter, keep):
    """A few rows of each group by themselves: the same bytes as among all of them."""
    c = Case(dev, sizes, hidden, inter, 4, True)
    h, hs, kept, ks = c.run_forward(keep)
    c.pos = None
    grad, q, qs, dw = c.run_backward(kept, ks)
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
        grad1, q1, qs1, dw1 = ep.ep_grouped_swiglu_backward(*c.dq, *c.down_t, kept1, ks1, off, rows=rows, rows_div=4,
                                                            weights=c.weights)
        assert all(torch.equal(a, b) for a, b in zip(
            _bytes(grad1, q1, qs1, dw1), _bytes(grad[at], q.view(torch.uint8)[at], qs[at], dw[at]))), count


def _held(v):
    """Float64 rows as 8 bits hold them."""
    t = S.blocks(v)
    unit = torch.exp2(S.scale_code(t.abs().amax(2)) - 127)[:, :, None]
    return (S.round_fp8(t / unit) * unit).flatten(1)[:, :v.shape[1]]


@pytest.mark.parametrize("sizes,hidden,inter", SHAPES[3:], ids=_name)
def test_outputs_are_off_by_little_more_than_their_rounding(dev, sizes, hidden, inter):
    """The products of h and of the 8-bit gradients, in norm, against their definition in 64 bits.

    A sum off by 2^-18 of a value passes a border of the 8 bits (steps of 2^-4 at most) once in 2^13 values; the output
    is off by 2^-6.5 2^-4 = 7e-4 then, beside 1.7e-3 of its own rounding to bf16: 1.1 times that, and 1.5 are granted, as
    rows are not of one size.  (Sums off by 2^-14 would make it 3e-3.)"""
    c = Case(dev, sizes, hidden, inter, 4, True)
    rng = np.random.default_rng(1)
    G = len(sizes)
    draw = lambda n, k: torch.from_numpy((rng.normal(0, 1, (G, n, k)) / np.sqrt(k)).astype(np.float32)).to(dev)  # noqa: E731
    wide = -(-inter // 128) * 128
    down, back = ep.ep_quant_blocks(draw(hidden, inter)), ep.ep_quant_blocks(draw(hidden, 2 * wide))
    back[0].view(torch.uint8).view(G, hidden, 2, wide)[:, :, :, inter:] = 0
    x, dy = S.values(*c.xq)[:, :hidden], S.values(*c.dq)[:, :hidden]
    y = torch.zeros((c.M, hidden), dtype=torch.float64, device=dev)
    dx = torch.zeros_like(y)
    h, hs, kept, ks = c.run_forward(BF16)
    grad, q, qs, _ = c.run_backward(kept, ks)
    for _, e, at, t, w in c._per_group((), 0):
        if e is None:
            break
        g, u = (x[t] @ S.matrix(v[e], s[e], hidden).t() for v, s in (c.gate, c.up))
        y[at] = _held(w * g * torch.sigmoid(g) * u) @ S.matrix(down[0][e], down[1][e], inter).t()
        d = dy[t] @ S.matrix(c.down_t[0][e], c.down_t[1][e], hidden).t()
        g, u = (v[at].double() for v in _split(kept, inter, inter))
        s = torch.sigmoid(g)
        dg, du = w * d * u * s * (1 + g * (1 - s)), w * d * g * s
        m = S.matrix(back[0][e], back[1][e], 2 * wide)
        dx[at] = _held(dg) @ m[:, :inter].t() + _held(du) @ m[:, wide:wide + inter].t()
    for name, got, want in (("y", ep.ep_grouped_matmul(h, hs, *down, c.offsets), y),
                            ("dx", ep.ep_grouped_matmul(q, qs, *back, c.offsets), dx)):
        own = float((want.float().to(BF16).double() - want).norm())
        assert float((got.double() - want).norm()) <= 1.5 * own, (name, float((got.double() - want).norm()) / own)


@pytest.mark.parametrize("sizes,hidden,inter", SHAPES, ids=_name)
def test_sums_of_8_bits_where_asked(dev, sizes, hidden, inter):
    """sums8: what is kept in bf16 has ep_grouped_matmul's sums, bit for bit, and h and the gradients lie within their
    bound."""
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
    r = c.backward(*(v.double() for v in _split(kept, inter, inter)))
    grad, q, qs, dw = c.run_backward(kept, None, sums8=True)
    wide, n = -(-inter // 128) * 128, -(-inter // 128)
    for name, got, side in zip(("dg", "du"), _split(grad, inter, inter), (0, 1)):
        S.check_bf16(got, r[name], r["e" + name], name)
        scale = torch.full((c.M, -(-n // 4) * 4), 127, dtype=torch.uint8, device=dev)
        scale[:, :n] = qs[:, side * n:(side + 1) * n]
        S.check_fp8(q[:, side * wide:(side + 1) * wide], scale, r[name], r["e" + name], name + " in 8 bits")
    pos = c.pos.long()
    want, e = (torch.where(pos >= 0, v[pos.clamp(min=0)], 0.0)
               for v in (r["dw"].sum(1), r["edw"].sum(1) + (128 + n) * 2.0 ** -24 * r["dw"].abs().sum(1)))
    assert ((dw.double() - want).abs() <= e).all()
    grad1, q1, qs1, dw1 = ep.ep_grouped_swiglu_backward(*c.dq, *c.down_t, kept1, None, off, rows=c.rows[at:at + 1],
                                                        rows_div=4, weights=c.weights, sums8=True)
    assert all(torch.equal(a[0], b[at]) for a, b in zip(_bytes(grad1, q1, qs1), _bytes(grad, q, qs)))
    if c.pair[at] >= 0:
        assert dw1[0] == dw[int(c.pair[at])]


@pytest.mark.parametrize("sums8", [False, True])
def test_the_layer_takes_the_callers_sums(dev, monkeypatch, sums8):
    """Both passes of a step have the sums that run_layer_train was given; fp32's unless asked."""
    from moe_expert_load_layer_amd import layer as module
    from test_gpu_layer_train import Setup
    seen, real = [], ep.lib()

    class Library:
        def __getattr__(self, name):
            call = getattr(real, name)
            if name not in ("ep_grouped_swiglu", "ep_grouped_swiglu_backward"):
                return call

            def spied(p, stream):
                seen.append((name, p._obj.sums8))
                return call(p, stream)
            return spied

    monkeypatch.setattr(module, "lib", Library)
    s = Setup(dev, 8, 4, 1, 300, 512, 640)
    k = dict(sums8=True) if sums8 else {}
    r = ep.run_layer_train(s.x, s.logits, 4, s.layout, s.experts, s.slots, **k)
    g = ep.run_layer_backward(r, s.dout, s.layout, s.back, s.back_slots)
    assert seen == [("ep_grouped_swiglu", int(sums8)), ("ep_grouped_swiglu_backward", int(sums8))]
    assert all(torch.isfinite(t.float()).all() for t in (r["out"], g["x"], g["logits"], g["gate_up"], g["down"]))
