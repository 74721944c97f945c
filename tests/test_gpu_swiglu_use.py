"""The gated block and the weight gradient of 8-bit rows in use: captured and replayed, on another stream, beside each
other, with infinities and NaN, with offsets that fall, with buffers that others surround, past 2^31 elements."""
import numpy as np
import pytest
import torch

import swiglu_ref as S
from test_gpu_stream_memory import _behind
from test_gpu_swiglu import BF16, FP8, Case

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _step(c, stream=None, keep=FP8):
    """All three operators in a row -> their outputs as byte tensors."""
    h, hs, kept, ks = c.run_forward(keep, stream=stream)
    grad, q, qs, dw = c.run_backward(kept, ks, stream=stream)
    w1 = ep.ep_grouped_wgrad_mixed(grad, *c.xq, c.offsets, cols=c.hidden, x_rows=c.rows, rows_div=c.div, stream=stream)
    w2 = ep.ep_grouped_wgrad_mixed(c.dy, h, hs, c.offsets, cols=c.inter, dy_rows=c.rows, rows_div=c.div, stream=stream)
    return [t.view(torch.uint8) for t in (h, hs, kept) + ((ks,) if ks is not None else ()) + (grad, q, qs, dw, w1, w2)]


def _same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


SIZES = [([150, 0, 201], 300, 200), ([3, 9], 513, 129)]


@pytest.mark.parametrize("sizes,hidden,inter", SIZES)
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_captured_and_replayed(dev, sizes, hidden, inter, keep):
    c = Case(dev, sizes, hidden, inter, 4, True, 5)
    eager = _step(c, keep=keep)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):          # two graphs of the same leaves
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _step(c, keep=keep)
        graphs.append((graph, out))
    for turn in range(4):
        for graph, out in graphs:
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert _same(out, eager), turn
        assert _same(_step(c, keep=keep), eager)
    # other inputs in the same places
    other = Case(dev, sizes, hidden, inter, 4, True, 5, seed=1)
    for mine, theirs in zip((c.xq[0], c.xq[1], c.dq[0], c.dq[1], c.weights, c.dy),
                            (other.xq[0], other.xq[1], other.dq[0], other.dq[1], other.weights, other.dy)):
        mine.copy_(theirs)
    fresh = _step(c, keep=keep)
    for graph, out in graphs:
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out, fresh)
    assert not _same(fresh, eager)


def test_on_a_stream_behind_other_work(dev):
    c = Case(dev, [40, 33, 0, 60], 260, 130, 4, True, 3)
    want = _step(c)
    torch.cuda.synchronize()
    assert _same(_behind(dev, lambda s: _step(c, s)), want)


def test_two_at_once(dev):
    a, b = Case(dev, [600, 500], 512, 256, 4, True), Case(dev, [90, 700, 33], 640, 384, 8, False, 9)
    want = [_step(a), _step(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [_step(c, s) for c, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert _same(got[0], want[0]) and _same(got[1], want[1])


def test_not_finite(dev):
    """An infinity or NaN stays in its token's rows, and out of their other blocks' scales."""
    c = Case(dev, [50, 47], 256, 384, 2, False)
    clean = _step(c)
    row = int(np.nonzero(c.pair // c.div == 5)[0][0])
    mine = torch.from_numpy(c.pair // c.div == 5).to(dev)
    for bad in (float("nan"), float("inf")):
        for which in ("x", "dy"):
            keep = getattr(c, which).clone()
            getattr(c, which)[5, 17] = bad
            c.xq, c.dq = ep.ep_quant_rows(c.x), ep.ep_quant_rows(c.dy)
            h, hs, kept, ks = c.run_forward(FP8)
            grad, q, qs, dw = c.run_backward(kept, ks)
            for i, t in enumerate((h, hs, kept, ks, grad, q, qs)):
                t = t.view(torch.uint8)
                assert torch.equal(t[~mine], clean[i].view(t.shape)[~mine]), (bad, which, i)
            if which == "x":
                assert torch.isnan(h.float()[row]).all() and (hs[row, :3] == 1).all()
            assert torch.isnan(q.float()[row]).all() and torch.isnan(grad.float()[row]).all()
            other = torch.ones_like(dw, dtype=torch.bool)
            other[5 * c.div:6 * c.div] = False
            assert torch.equal(dw[other], clean[7].view(torch.float32)[other])
            getattr(c, which).copy_(keep)
    c.xq, c.dq = ep.ep_quant_rows(c.x), ep.ep_quant_rows(c.dy)
    # an infinite weight: h and the gradients are infinite (NaN in 8 bits), g and u are as they were
    c.weights[int(c.pair[row])] = float("inf")
    h, hs, kept, ks = c.run_forward(FP8)
    assert torch.equal(kept.view(torch.uint8).flatten(), clean[2].flatten())
    assert torch.isnan(h.float()[row]).any() and (hs[row, :3] == 1).all()
    grad, q, qs, _ = c.run_backward(kept, ks)
    assert not torch.isfinite(grad.float()[row]).any() and torch.isfinite(grad.float()[row - 1]).all()
    # one infinity beside finite values: they keep their own scale
    c.weights.fill_(1.0)
    c.gate[0][:] = 0
    big = torch.full((384, 256), 0.0, device=dev)
    big[7] = 1e30
    c.up = ep.ep_quant_blocks(big.expand(2, -1, -1).contiguous())
    c.gate = c.up
    h, hs, _, _ = c.run_forward(None)
    # silu of -1e30 and less is 0, of 1e30 and more infinite once multiplied by u
    token = torch.from_numpy(c.pair // c.div).to(dev)
    large = S.values(*c.xq)[token].sum(1) > 0
    assert torch.equal(torch.isnan(h.float()[:, 7]), large) and (h.float()[~large, 7] == 0).all()
    assert (h.float()[:, 8:] == 0).all() and (hs[:, :3] == 1).all()


def test_offsets_that_fall_or_lie_outside(dev):
    """Such offsets are brought into the buffer: rows of no group may hold anything, those around it are untouched."""
    c = Case(dev, [300, 200, 100], 256, 256, 0, False)
    wild = torch.tensor([-5, 450, 120, 9000], dtype=torch.int32, device=dev)
    good, c.offsets = c.offsets, wild
    M, I = c.M, 256
    parts = {}

    def inside(name, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        parts[name] = (torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=dev), n)
        return parts[name][0][2048:2048 + n].view(dtype).view(shape)
    h, hs, kept, ks = c.run_forward(FP8, h=inside("h", (M, I), FP8), h_scale=inside("hs", (M, 4), torch.uint8),
                                    kept=inside("kept", (M, 2 * I), FP8), kept_scale=inside("ks", (M, 4), torch.uint8))
    grad, q, qs, dw = c.run_backward(kept, ks, grad=inside("grad", (M, 2 * I), BF16), q=inside("q", (M, 2 * I), FP8),
                                     q_scale=inside("qs", (M, 4), torch.uint8),
                                     grad_weights=inside("dw", (M,), torch.float32))
    ep.ep_grouped_wgrad_mixed(c.dy, h, hs, wild, cols=I, out=inside("dw1", (3, 256, I), torch.float32))
    torch.cuda.synchronize()
    for name, (flat, n) in parts.items():
        assert (flat[:2048] == 0xA5).all() and (flat[2048 + n:] == 0xA5).all(), name
    # the first group, rows 0 .. 449, is as it would be alone
    c.offsets = torch.tensor([0, 450, 450, 450], dtype=torch.int32, device=dev)
    alone = c.run_forward(None)[0]
    assert torch.equal(h.view(torch.uint8)[:120], alone.view(torch.uint8)[:120])
    c.offsets = good


def test_rows_and_groups_none(dev):
    """No rows at all, and one group without offsets."""
    c = Case(dev, [0, 0], 256, 200, 0, False)
    h, hs, kept, ks = c.run_forward(FP8)
    assert h.shape == (0, 256) and kept.shape == (0, 512)
    grad, q, _, dw = c.run_backward(kept, ks)
    assert grad.shape == (0, 400) and dw.shape == (0,)
    assert (ep.ep_grouped_wgrad_mixed(c.dy, h, hs, c.offsets, cols=200) == 0).all()
    d = Case(dev, [77], 256, 200, 0, False)
    with_ = _step(d)
    d.offsets = None
    assert _same(_step(d), with_)


@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_past_31_bits(dev, keep):
    """More than 2^31 elements of what is kept and of the gradients, a few of the last rows checked."""
    M, hidden, inter, tokens = 560_001, 128, 2048, 5000
    g = torch.Generator(device=dev).manual_seed(9)
    x = torch.randn((tokens, hidden), generator=g, device=dev).to(BF16)
    dy = (1e-2 * torch.randn((tokens, hidden), generator=g, device=dev)).to(BF16)
    w = lambda n, k: torch.randn((2, n, k), generator=g, device=dev) * k ** -0.5  # noqa: E731
    gate, up = ep.ep_quant_blocks(w(inter, hidden)), ep.ep_quant_blocks(w(inter, hidden))
    down = ep.ep_quant_blocks(w(hidden, inter), transpose=True)
    rows = torch.randint(0, tokens, (M,), generator=g, device=dev, dtype=torch.int32)
    weights = torch.rand(tokens, generator=g, device=dev)
    off = torch.tensor([0, 1000, M], dtype=torch.int32, device=dev)
    xq, dq = ep.ep_quant_rows(x), ep.ep_quant_rows(dy)
    h, hs, kept, ks = ep.ep_grouped_swiglu(*xq, *gate, *up, off, rows=rows, weights=weights, keep=keep)
    grad, q, qs, dw = ep.ep_grouped_swiglu_backward(*dq, *down, kept, ks, off, rows=rows, weights=weights,
                                                    pos=torch.arange(M, device=dev, dtype=torch.int32).flip(0))
    assert kept.numel() > 2 ** 31 and grad.numel() > 2 ** 31
    few = slice(M - 40, M)
    t = rows[few].long()
    xv, dv, w = S.values(*xq), S.values(*dq), weights[t].double()[:, None]
    g, eg, u, eu, hw, eh = S.forward(xv[t], S.matrix(gate[0][1], gate[1][1], hidden), S.matrix(up[0][1], up[1][1], hidden), w)
    S.check_fp8(h[few], hs[few], hw, eh, "h")
    if keep is FP8:
        full = S.values(kept[few], ks[few])
        for name, at, want, e in (("g", 0, g, eg), ("u", 1, u, eu)):
            S.check_fp8(kept[few, at * inter:(at + 1) * inter], ks[few, at * 16:(at + 1) * 16], want, e, name)
    else:
        full = kept[few].double()
        S.check_bf16(kept[few], torch.cat([g, u], 1), torch.cat([eg, eu], 1), "kept")
    back = S.matrix(down[0][1], down[1][1], hidden)
    d, ed = dv[t] @ back.t(), S.DROPPED * (dv[t].abs() @ back.abs().t())
    dg, edg, du, edu, terms, et = S.backward(d, ed, full[:, :inter], full[:, inter:], w)
    S.check_bf16(grad[few], torch.cat([dg, du], 1), torch.cat([edg, edu], 1), "gradients")
    for at, want, e in ((0, dg, edg), (1, du, edu)):
        S.check_fp8(q[few, at * inter:(at + 1) * inter], qs[few, at * 16:(at + 1) * 16], want, e, "in 8 bits")
    bound = et.sum(1) + (128 + 16) * 2.0 ** -24 * terms.abs().sum(1)
    assert ((dw[:40].flip(0).double() - terms.sum(1)).abs() <= bound).all()
    if keep is FP8:
        return
    got = ep.ep_grouped_wgrad_mixed(grad, *xq, off, cols=hidden, x_rows=rows)[1]
    want, size = torch.zeros(2 * inter, hidden, dtype=torch.float64, device=dev), torch.zeros_like(got, dtype=torch.float64)
    for at in range(1000, M, 100_000):
        i = slice(at, min(M, at + 100_000))
        a, b = grad[i].double(), xv[rows[i].long()]
        want += a.t() @ b
        size += a.abs().t() @ b.abs()
    assert ((got.double() - want).abs() <= (M + 8) * 2.0 ** -24 * size).all()
