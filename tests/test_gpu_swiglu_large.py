"""The gated block's largest tiles, with either kind of sums: workgroups that take tile after tile, ragged rows and
columns, three blocks of terms and more; infinities and NaN, falling offsets, replay, two streams, more than 2^31
elements."""
import numpy as np
import pytest
import torch

import swiglu_ref as S
from test_gpu_swiglu import BF16, FP8, Case, _split

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")

# 67 x 16 tiles of 256 rows forward, 67 x 8 of 256 x 256 backward; four blocks of terms, part rows and columns
LARGE = ([9000, 8001, 0], 400, 2020)
SUMS = pytest.mark.parametrize("sums8", [False, True], ids=["fp32", "8bit"])
KEEP = pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _part(scales, at, n, M):
    """The scale bytes of one of the two blocks that lie side by side, as rows of its own."""
    out = torch.full((M, -(-n // 4) * 4), 127, dtype=torch.uint8, device=scales.device)
    out[:, :n] = scales[:, at * n:(at + 1) * n]
    return out


@SUMS
@KEEP
@pytest.mark.parametrize("extra", [0, 300])
def test_values(dev, keep, sums8, extra):
    sizes, hidden, inter = LARGE
    c = Case(dev, sizes, hidden, inter, 8, True, extra)
    h, hs, kept, ks = c.run_forward(keep, sums8=sums8)
    r = c.forward()
    S.check_fp8(h, hs, r["h"], r["eh"], "h")
    wide, n = -(-inter // 128) * 128, -(-inter // 128)
    for name, at in (("g", 0), ("u", 1)):
        if keep is FP8:
            S.check_fp8(kept[:, at * wide:(at + 1) * wide], _part(ks, at, n, c.M), r[name], r["e" + name], name)
        else:
            S.check_bf16(kept[:, at * inter:(at + 1) * inter], r[name], r["e" + name], name)
    kg, ku = _split(S.values(kept, ks) if keep is FP8 else kept.double(), inter, wide if keep is FP8 else inter)
    r = c.backward(kg, ku)
    grad, q, qs, dw = c.run_backward(kept, ks, sums8=sums8)
    for name, got, at in zip(("dg", "du"), _split(grad, inter, inter), (0, 1)):
        S.check_bf16(got, r[name], r["e" + name], name)
        S.check_fp8(q[:, at * wide:(at + 1) * wide], _part(qs, at, n, c.M), r[name], r["e" + name], name + " in 8 bits")
    at = c.pos.long()
    want, e = (torch.where(at >= 0, v[at.clamp(min=0)], 0.0)
               for v in (r["dw"].sum(1), r["edw"].sum(1) + (128 + n) * 2.0 ** -24 * r["dw"].abs().sum(1)))
    assert ((dw.double() - want).abs() <= e).all()
    none = torch.from_numpy(np.where(np.arange(c.M) < c.total, c.pair, -1) < 0).to(dev)
    assert (h.view(torch.uint8)[none] & 127 == 0).all() and (hs[none][:, :n] == 1).all()
    assert (kept[none].double() == 0).all() and (grad[none] == 0).all() and (q[none].double() == 0).all()


def _step(c, sums8, keep=FP8, stream=None):
    h, hs, kept, ks = c.run_forward(keep, stream=stream, sums8=sums8)
    grad, q, qs, dw = c.run_backward(kept, ks, stream=stream, sums8=sums8)
    return [t.view(torch.uint8) for t in (h, hs, kept, ks, grad, q, qs, dw) if t is not None]


def _same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@SUMS
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["x", "dy"])
def test_not_finite(dev, sums8, bad, which):
    sizes, hidden, inter = LARGE
    c = Case(dev, sizes, hidden, inter, 8, True)
    clean = _step(c, sums8)
    token = int(c.pair[c.pair >= 0][4000]) // 8
    mine = torch.from_numpy((c.pair >= 0) & (c.pair // 8 == token)).to(dev)
    getattr(c, which)[token, 170] = bad
    c.xq, c.dq = ep.ep_quant_rows(c.x), ep.ep_quant_rows(c.dy)
    got = _step(c, sums8)
    for i, (a, b) in enumerate(zip(got[:-1], clean[:-1])):
        assert torch.equal(a[~mine], b[~mine]), i
    dw, was = (v[-1].view(torch.float32) for v in (got, clean))
    pairs = torch.arange(len(dw), device=dev) // 8 == token
    assert torch.equal(dw[~pairs], was[~pairs]) and torch.isnan(dw[pairs & (c.pos >= 0)]).all()
    width = 2048
    assert torch.isnan(got[5].view(FP8).float()[mine][:, :inter]).all()
    assert torch.isnan(got[5].view(FP8).float()[mine][:, width:width + inter]).all()
    if which == "x":
        assert torch.isnan(got[0].view(FP8).float()[mine][:, :inter]).all() and (got[1][mine][:, :16] == 1).all()


@SUMS
@KEEP
def test_offsets_that_fall_or_lie_outside(dev, keep, sums8):
    """Brought into the buffers: nothing around them is touched, and the first group is as it would be alone."""
    sizes, hidden, inter = LARGE
    c = Case(dev, sizes, hidden, inter, 0, False)
    M, wide = c.M, -(-inter // 128) * 128
    parts = {}

    def inside(name, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        parts[name] = (torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=dev), n)
        return parts[name][0][2048:2048 + n].view(dtype).view(shape)

    alone_offsets = torch.tensor([0, 12000, 12000, 12000], dtype=torch.int32, device=dev)
    c.offsets = torch.tensor([-5, 12000, 3000, 90000], dtype=torch.int32, device=dev)
    eight = keep is FP8
    kept_shape = (M, 2 * wide) if eight else (M, 2 * inter)
    sb, ksb = ep.ep_scale_stride(inter), ep.ep_scale_stride(2 * wide)
    h, hs, kept, ks = c.run_forward(keep, h=inside("h", (M, wide), FP8), h_scale=inside("hs", (M, sb), torch.uint8),
                                    kept=inside("kept", kept_shape, keep),
                                    kept_scale=inside("ks", (M, ksb), torch.uint8) if eight else None, sums8=sums8)
    grad, q, qs, dw = c.run_backward(kept, ks, grad=inside("grad", (M, 2 * inter), BF16),
                                     q=inside("q", (M, 2 * wide), FP8), q_scale=inside("qs", (M, ksb), torch.uint8),
                                     grad_weights=inside("dw", (M,), torch.float32), sums8=sums8)
    torch.cuda.synchronize()
    for name, (flat, n) in parts.items():
        assert (flat[:2048] == 0xA5).all() and (flat[2048 + n:] == 0xA5).all(), name
    c.offsets = alone_offsets
    alone = c.run_forward(keep, sums8=sums8)
    assert torch.equal(h.view(torch.uint8)[:3000], alone[0].view(torch.uint8)[:3000])
    assert torch.equal(kept.view(torch.uint8)[:3000], alone[2].view(torch.uint8)[:3000])
    back = c.run_backward(alone[2], alone[3], sums8=sums8)
    assert torch.equal(q.view(torch.uint8)[:3000], back[1].view(torch.uint8)[:3000])
    assert torch.equal(grad[:3000], back[0][:3000])


@SUMS
@KEEP
def test_captured_and_replayed(dev, keep, sums8):
    sizes, hidden, inter = LARGE
    c = Case(dev, sizes, hidden, inter, 8, True, 5)
    eager = _step(c, sums8, keep)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _step(c, sums8, keep)
        graphs.append((graph, out))
    for turn in range(3):
        for graph, out in graphs:
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert _same(out, eager), turn
        assert _same(_step(c, sums8, keep), eager)


def test_two_at_once(dev):
    """Both kinds of sums on streams of their own."""
    sizes, hidden, inter = LARGE
    a, b = Case(dev, sizes, hidden, inter, 8, True), Case(dev, [5000, 4100], 700, 1400, 4, False, 9)
    want = [_step(a, False), _step(b, True)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [_step(c, s8, FP8, s) for c, s8, s in zip((a, b), (False, True), streams)]
        torch.cuda.synchronize()
        assert _same(got[0], want[0]) and _same(got[1], want[1])


@SUMS
@KEEP
def test_past_31_bits(dev, keep, sums8):
    """More than 2^31 elements of what is kept and of the gradients, with tiles taken one after the other."""
    M, hidden, inter, tokens = 560_001, 400, 2048, 5000
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
    h, hs, kept, ks = ep.ep_grouped_swiglu(*xq, *gate, *up, off, rows=rows, weights=weights, keep=keep, sums8=sums8)
    grad, q, qs, dw = ep.ep_grouped_swiglu_backward(*dq, *down, kept, ks, off, rows=rows, weights=weights, sums8=sums8)
    assert kept.numel() > 2 ** 31 and grad.numel() > 2 ** 31
    few = torch.cat([torch.arange(a, a + 40, device=dev) for a in (0, 980, M // 2, 524_260, M - 40)])
    for e, at in ((0, few[few < 1000]), (1, few[few >= 1000])):
        t = rows[at].long()
        xv, dv, wt = S.values(*xq)[:, :hidden], S.values(*dq)[:, :hidden], weights[t].double()[:, None]
        mg, mu = (S.matrix(m[0][e], m[1][e], hidden) for m in (gate, up))
        vg, eg, vu, eu, vh, eh = S.forward(xv[t], mg, mu, wt)
        S.check_fp8(h[at], hs[at], vh, eh, "h")
        if keep is FP8:
            full = S.values(kept[at], ks[at])
            for side, want, b in ((0, vg, eg), (1, vu, eu)):
                S.check_fp8(kept[at, side * inter:(side + 1) * inter], ks[at, side * 16:(side + 1) * 16], want, b, "kept")
        else:
            full = kept[at].double()
            S.check_bf16(kept[at], torch.cat([vg, vu], 1), torch.cat([eg, eu], 1), "kept")
        back = S.matrix(down[0][e], down[1][e], hidden)
        d, ed = dv[t] @ back.t(), S.DROPPED * (dv[t].abs() @ back.abs().t())
        dg, edg, du, edu, terms, et = S.backward(d, ed, full[:, :inter], full[:, inter:], wt)
        S.check_bf16(grad[at], torch.cat([dg, du], 1), torch.cat([edg, edu], 1), "gradients")
        for side, want, b in ((0, dg, edg), (1, du, edu)):
            S.check_fp8(q[at, side * inter:(side + 1) * inter], qs[at, side * 16:(side + 1) * 16], want, b, "in 8 bits")
        bound = et.sum(1) + (128 + 16) * 2.0 ** -24 * terms.abs().sum(1)
        assert ((dw[at].double() - terms.sum(1)).abs() <= bound).all()
