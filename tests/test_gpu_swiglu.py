"""The gated feed-forward block over groups of rows, forward and backward, and the weight gradient of rows in 8 bits,
against plain 64-bit forms (swiglu_ref.py has the bounds).  Weight gradient: products of a bf16 and an e4m3 value are
exact in fp32, additions rounded: (m + 8) 2^-24 sum |dy x| at the most."""
import numpy as np
import pytest
import torch

import swiglu_ref as S

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")

FP8, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _rows(rng, M, K, dev, std=1.0):
    a = rng.normal(0, std, (M, K)) * np.exp(0.5 * rng.normal(0, 1, (M, 1)))
    a[:, rng.random(K) < 0.02] *= 20
    out = torch.empty((M, K), dtype=BF16, device=dev)
    return out.copy_(torch.from_numpy(a.astype(np.float32)).to(dev))


class Case:
    """A block's inputs: `sizes` of the groups, `div` pairs a token (0: rows in order), some positions without a pair."""

    def __init__(self, dev, sizes, hidden, inter, div=0, masked=False, extra=0, weights=True, seed=0):
        rng = np.random.default_rng(seed + 7 * hidden + inter)
        self.sizes, self.hidden, self.inter, self.div = sizes, hidden, inter, max(1, div)
        self.total, self.M, G = sum(sizes), sum(sizes) + extra, len(sizes)
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=dev)
        self.rows = self.pos = None
        self.pair = np.arange(self.M)
        self.tokens = self.M
        if div:
            self.tokens = max(1, -(-self.M // div))
            self.pair = rng.permutation(self.M)
            if masked:
                self.pair = np.where(rng.random(self.M) < 0.2, -1, self.pair)
                self.pair[rng.integers(self.M)] = self.tokens * div + 5     # past the tokens
            self.rows = torch.from_numpy(self.pair.astype(np.int32)).to(dev)
            self.pair = np.where(self.pair >= self.tokens * div, -1, self.pair)
            pos = np.full(self.tokens * div, -1)
            pos[self.pair[self.pair >= 0]] = np.nonzero(self.pair >= 0)[0]
            self.pos = torch.from_numpy(pos.astype(np.int32)).to(dev)
        self.x, self.dy = _rows(rng, self.tokens, hidden, dev), _rows(rng, self.tokens, hidden, dev, 1e-2)
        w = lambda n, k: torch.from_numpy((rng.normal(0, 1, (G, n, k)) / np.sqrt(k)).astype(np.float32)).to(dev)  # noqa: E731
        gate, up, down = w(inter, hidden), w(inter, hidden), w(hidden, inter)
        self.gate, self.up = ep.ep_quant_blocks(gate), ep.ep_quant_blocks(up)
        self.down_t = ep.ep_quant_blocks(down, transpose=True)
        count = self.M if self.rows is None else self.tokens * self.div
        self.weights = torch.from_numpy(rng.random(count).astype(np.float32)).to(dev) if weights else None
        if weights:
            self.weights[::5] = 0
            self.weights[1::7] *= -3
        self.xq, self.dq = ep.ep_quant_rows(self.x), ep.ep_quant_rows(self.dy)

    def groups(self):
        """(group, its positions that a pair takes)."""
        at = 0
        for g, n in enumerate(self.sizes):
            i = np.arange(at, at + n)
            yield g, torch.from_numpy(i[self.pair[i] >= 0]).to(self.x.device)
            at += n

    def _per_group(self, what, width):
        out = {k: torch.zeros((self.M, width), dtype=torch.float64, device=self.x.device) for k in what}
        pair = torch.from_numpy(self.pair).to(self.x.device)
        for g, at in self.groups():
            if len(at):
                p = pair[at]
                w = torch.ones((len(at), 1), device=self.x.device).double() if self.weights is None else \
                    self.weights[p].double()[:, None]
                yield out, g, at, p // self.div, w
        yield out, None, None, None, None

    def forward(self):
        x = S.values(*self.xq)[:, :self.hidden]
        names = ("g", "eg", "u", "eu", "h", "eh")
        for out, g, at, t, w in self._per_group(names, self.inter):
            if g is None:
                return out
            gate, up = (S.matrix(q[g], s[g], self.hidden) for q, s in (self.gate, self.up))
            for name, v in zip(names, S.forward(x[t], gate, up, w)):
                out[name][at] = v

    def backward(self, kg, ku):
        dy = S.values(*self.dq)[:, :self.hidden]
        names = ("dg", "edg", "du", "edu", "dw", "edw")
        for out, g, at, t, w in self._per_group(names, self.inter):
            if g is None:
                return out
            down = S.matrix(self.down_t[0][g], self.down_t[1][g], self.hidden)
            d, ed = dy[t] @ down.t(), S.DROPPED * (dy[t].abs() @ down.abs().t())
            for name, v in zip(names, S.backward(d, ed, kg[at], ku[at], w)):
                out[name][at] = v

    def run_forward(self, keep=None, **k):
        return ep.ep_grouped_swiglu(*self.xq, *self.gate, *self.up, self.offsets, rows=self.rows, rows_div=self.div,
                                    weights=self.weights, keep=keep, **k)

    def run_backward(self, kept, kept_scale, **k):
        return ep.ep_grouped_swiglu_backward(*self.dq, *self.down_t, kept, kept_scale, self.offsets, rows=self.rows,
                                             rows_div=self.div, weights=self.weights, pos=self.pos, **k)


def _split(t, inter, wide):
    return t[:, :inter], t[:, wide:wide + inter]


# sizes of groups, hidden, inter, pairs a token, masked, rows past the groups, weights
SHAPES = [
    ([1], 128, 128, 0, False, 0, True), ([3], 64, 1, 0, False, 0, False), ([2, 0, 5], 130, 127, 2, False, 0, True),
    ([9, 40, 0, 1], 257, 129, 4, True, 7, True), ([64, 63], 1000, 300, 8, False, 0, False),
    ([1, 1, 1, 1], 768, 256, 4, True, 0, True), ([100, 130], 513, 255, 0, False, 3, True),
    ([200, 97, 128], 700, 640, 8, True, 0, True), ([128, 300], 2048, 384, 0, False, 0, True),
    ([4100], 200, 1500, 4, True, 0, True), ([2500, 1700, 0], 650, 1800, 8, False, 90, True),
    ([5000], 1024, 1280, 0, False, 0, False), ([30000, 22000, 0], 99, 103, 8, False, 0, True),
    ([26000, 30001], 640, 130, 4, True, 5, True), ([700, 801], 640, 1500, 4, True, 3, True),
    ([1501], 400, 1450, 0, False, 0, True), ([100] * 15 + [61], 600, 1401, 8, True, 0, True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("keep", [None, BF16, FP8], ids=["none", "bf16", "fp8"])
def test_forward(dev, shape, keep):
    sizes, hidden, inter, div, masked, extra, weighted = shape
    c = Case(dev, sizes, hidden, inter, div, masked, extra, weighted)
    r = c.forward()
    wide = -(-inter // 128) * 128
    fill = lambda shape, dtype: torch.full(shape, 0x55, dtype=torch.uint8, device=dev).view(dtype)  # noqa: E731
    h, hs = fill((c.M, wide), FP8), fill((c.M, ep.ep_scale_stride(inter)), torch.uint8)
    h, hs, kept, ks = c.run_forward(keep, h=h, h_scale=hs)
    S.check_fp8(h, hs, r["h"], r["eh"], "h")
    if keep is FP8:
        # two blocks of their own: g, zeros, u, zeros
        n = wide // 128
        for name, at in (("g", 0), ("u", 1)):
            scale = torch.full((c.M, -(-n // 4) * 4), 127, dtype=torch.uint8, device=dev)
            scale[:, :n] = ks[:, at * n:(at + 1) * n]
            S.check_fp8(kept[:, at * wide:(at + 1) * wide], scale, r[name], r["e" + name], name)
        assert (ks[:, 2 * n:] == 127).all()
    elif keep is BF16:
        for name, got in zip(("g", "u"), _split(kept, inter, inter)):
            S.check_bf16(got, r[name], r["e" + name], name)
    else:
        assert kept is None and ks is None
    # rows without a pair and rows past the groups are rows of zeros
    none = torch.from_numpy(np.where(np.arange(c.M) < c.total, c.pair, -1) < 0).to(dev)
    assert (h.view(torch.uint8)[none] & 127 == 0).all() and (hs[none][:, :wide // 128] == 1).all()
    if kept is not None:
        assert (kept[none].double() == 0).all()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_backward(dev, shape, keep):
    sizes, hidden, inter, div, masked, extra, weighted = shape
    c = Case(dev, sizes, hidden, inter, div, masked, extra, weighted)
    _, _, kept, ks = c.run_forward(keep)
    wide = -(-inter // 128) * 128
    full = S.values(kept, ks) if keep is FP8 else kept.double()
    kg, ku = _split(full, inter, wide if keep is FP8 else inter)
    r = c.backward(kg, ku)
    if not weighted:
        c.pos = None
    grad, q, qs, dw = c.run_backward(kept, ks)
    n = wide // 128
    for name, got, at in zip(("dg", "du"), _split(grad, inter, inter), (0, 1)):
        S.check_bf16(got, r[name], r["e" + name], name)
        scale = torch.full((c.M, -(-n // 4) * 4), 127, dtype=torch.uint8, device=dev)
        scale[:, :n] = qs[:, at * n:(at + 1) * n]
        S.check_fp8(q[:, at * wide:(at + 1) * wide], scale, r[name], r["e" + name], name + " in 8 bits")
    assert (qs[:, 2 * n:] == 127).all()
    none = torch.from_numpy(np.where(np.arange(c.M) < c.total, c.pair, -1) < 0).to(dev)
    assert (grad[none] == 0).all() and (q[none].double() == 0).all()
    if not weighted:
        assert dw is None
        return
    by_row, bound = r["dw"].sum(1), r["edw"].sum(1) + (128 + n) * 2.0 ** -24 * r["dw"].abs().sum(1)
    if c.pos is None:
        want, e = by_row, bound
    else:
        at = c.pos.long()
        want, e = (torch.where(at >= 0, v[at.clamp(min=0)], 0.0) for v in (by_row, bound))
    assert ((dw.double() - want).abs() <= e).all()
    half = c.run_backward(kept, ks, weights_dtype=BF16)[3]
    assert torch.equal(half, dw.to(BF16))


@pytest.mark.parametrize("sizes,inter", [([300, 211], 256), ([3000, 2111], 256), ([3500, 2311], 384)], ids=str)
def test_fused_and_apart_agree(dev, sizes, inter):
    """The block in one product against the grouped product in bf16 and the step on its own: 2^-9 apart before the 8
    bits.  With many rows of many columns they have the same sums, rounded once; else exact sums against those: their
    bound and a rounding of each, 2^-8 of a value."""
    c = Case(dev, sizes, 640, inter, 4, weights=False)
    both = torch.cat([c.gate[0].view(torch.uint8), c.up[0].view(torch.uint8)], 1).view(FP8)
    apart = ep.ep_grouped_matmul(*c.xq, both, torch.cat([c.gate[1], c.up[1]], 1), c.offsets, rows=c.rows, rows_div=4)
    h, hs, kept, _ = c.run_forward(BF16)
    if inter > 256:
        assert torch.equal(kept, apart)
    else:
        r = c.forward()
        v, e = torch.cat([r["g"], r["u"]], 1).abs(), torch.cat([r["eg"], r["eu"]], 1)
        assert ((kept.double() - apart.double()).abs() <= e + 2 * 2.0 ** -8 * (v + e)).all()
    q, s = ep.ep_swiglu_quant(apart)
    one, two = S.values(h, hs), S.values(q, s)
    assert float((one - two).norm()) < 0.05 * float(two.norm())


WGRAD = [([1], 128, 128, "", False), ([2, 0, 5], 8, 1, "x", False), ([70, 33, 1], 264, 300, "dy", True),
         ([31, 32, 97], 300, 129, "x", True), ([128, 1, 400], 520, 260, "both", True), ([1000], 7, 500, "dy", False),
         ([385, 255], 511, 640, "", False), ([900, 700, 0, 30], 1032, 384, "x", True), ([40], 3, 77, "", False)]


@pytest.mark.parametrize("shape", WGRAD, ids=str)
@pytest.mark.parametrize("extra", [0, 11])
def test_wgrad_mixed(dev, shape, extra):
    sizes, N, K, gather, masked = shape
    rng = np.random.default_rng(N * K)
    total, div = sum(sizes), 3
    M = total + extra
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=dev)
    tokens = -(-M // div)
    pair = rng.permutation(M) if gather else np.arange(M)
    if masked:
        pair = np.where(rng.random(M) < 0.3, -1 - pair, pair)
        pair[0] = tokens * div + 2
    rows = torch.from_numpy(pair.astype(np.int32)).to(dev) if gather else None
    has = (pair >= 0) & (pair < tokens * div) if gather else np.ones(M, bool)
    count = lambda name: tokens if gather in (name, "both") else M  # noqa: E731
    dy, x = _rows(rng, count("dy"), N, dev), _rows(rng, count("x"), K, dev)
    q, s = ep.ep_quant_rows(x)
    junk = torch.from_numpy(np.nonzero(~has)[0]).to(dev)
    if gather == "x":
        dy[junk] = float("nan")             # rows that no pair takes are not read into the sum
    if gather == "dy":
        q.view(torch.uint8)[junk] = 0x7F
    G = len(sizes)
    out = torch.full((G, N, K), 5.0, device=dev)
    got = ep.ep_grouped_wgrad_mixed(dy, q, s, offsets, cols=K, dy_rows=rows if gather in ("dy", "both") else None,
                                    x_rows=rows if gather in ("x", "both") else None, rows_div=div, out=out)
    assert got is out
    xv, dv = S.values(q, s)[:, :K], dy.double()
    at = 0
    for g, n in enumerate(sizes):
        i = torch.from_numpy(np.arange(at, at + n)[has[at:at + n]]).to(dev)
        t = torch.from_numpy(pair).to(dev)[i] // div if gather else i
        a = dv[t if gather in ("dy", "both") else i]
        b = xv[t if gather in ("x", "both") else i]
        want, mag = a.t() @ b, a.abs().t() @ b.abs()
        assert ((got[g].double() - want).abs() <= (n + 8) * 2.0 ** -24 * mag).all(), g
        at += n


def test_wgrad_mixed_is_exact_on_whole_numbers(dev):
    """Small whole numbers under every scale that keeps the sums whole: bit for bit."""
    rng = np.random.default_rng(5)
    M, N, K = 300, 264, 384
    dy = torch.from_numpy(rng.integers(-4, 5, (M, N)).astype(np.float32)).to(BF16).to(dev)
    x = torch.from_numpy(rng.integers(-7, 8, (M, K)).astype(np.float32)).to(dev)
    x[:, :128] *= 2.0 ** torch.randint(0, 6, (M, 1), device=dev)
    q, s = ep.ep_quant_rows(x)
    got = ep.ep_grouped_wgrad_mixed(dy, q, s)[0]
    assert torch.equal(got.double(), dy.double().t() @ x.double())
    tiny = ep.ep_quant_rows(x * 2.0 ** -120)
    assert torch.equal(ep.ep_grouped_wgrad_mixed(dy, *tiny)[0], got * 2.0 ** -120)
