"""run_layer_train and run_layer_backward: a whole training step of the layer against the plain layer's gradients in 64
bits, by formula and by differences; replicas; padded tokens.

Against exact arithmetic on the same 8-bit weights and inputs the path rounds to 8 bits: dout, g, u, h and the inner
gradient, each by at most 2^-4 of a value and by 2^-4 / sqrt(3) * 0.72 = 2.6 % in the mean square.  At most four such
roundings lie on the way to any result (out: h; x: dout, g, u, the inner one; the matrices: three; the logits: dout, g, u,
and the difference from the weighted mean, which takes away at most as much as it leaves in these inputs): 5.2 % for
independent ones, 0.1 is asked."""
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


class Setup:
    def __init__(self, dev, E, ranks, spare, tokens, H, I, dtype=torch.float32, apart=False, masked=False):
        g = torch.Generator(device=dev).manual_seed(E + H)
        randn = lambda *s: torch.randn(s, generator=g, device=dev)     # noqa: E731
        self.layout = ep.Layout.create(E, [E // ranks] * ranks, list(range(E)), [spare] * ranks, device=dev)
        self.gate_up, self.down = randn(E, 2 * I, H) * H ** -0.5, randn(E, H, I) * I ** -0.5
        self.experts = ep.ExpertRows(E, H, I, dev, apart=apart).load(self.gate_up, self.down)
        self.back = ep.ExpertBackwardRows(E, H, I, dev).load(self.gate_up, self.down)
        n = self.layout.num_spare
        self.slots, self.back_slots = ep.ExpertRows(n, H, I, dev, apart=apart), ep.ExpertBackwardRows(n, H, I, dev)
        self.x = randn(ranks * tokens, H).to(BF16)
        self.logits = (randn(ranks * tokens, E) + 2 * torch.rand(E, generator=g, device=dev)).to(dtype)
        if masked:
            self.logits[3:5] = -float("inf")
        self.dout = (randn(ranks * tokens, H) * 1e-2).to(BF16)

    def step(self, k, keep=FP8):
        r = ep.run_layer_train(self.x, self.logits, k, self.layout, self.experts, self.slots, keep=keep)
        return r, ep.run_layer_backward(r, self.dout, self.layout, self.back, self.back_slots)


def _plain(s, ids, inter):
    """The layer on the 8-bit values, as a function of float64 leaves; `ids` fixed."""
    E, H = s.gate_up.shape[0], s.gate_up.shape[2]
    ex = s.experts
    gate = torch.stack([S.matrix(ex.gate[e], ex.gate_scale[e], H) for e in range(E)])
    up = torch.stack([S.matrix(ex.up[e], ex.up_scale[e], H) for e in range(E)])
    down = torch.stack([S.matrix(ex.down[e], ex.down_scale[e], inter) for e in range(E)])
    x = S.values(*ep.ep_quant_rows(s.x))[:, :H]
    leaves = [t.cpu().requires_grad_() for t in (x, s.logits.double(), gate, up, down)]
    ids = ids.cpu().long()

    def layer(x, logits, gate, up, down):
        out = torch.zeros_like(x)
        chosen = ids >= 0
        z = torch.where(chosen, logits.gather(1, ids.clamp(min=0)), torch.tensor(-1e30, dtype=torch.float64))
        w = torch.softmax(z, dim=1) * chosen
        for e in range(E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if len(t):
                a = x[t] @ gate[e].t()
                y = (torch.nn.functional.silu(a) * (x[t] @ up[e].t())) @ down[e].t()
                out = out.index_add(0, t, w[t, j][:, None] * y)
        return out
    return layer, leaves


def _apart(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


CASES = [dict(E=8, ranks=4, spare=1, tokens=48, H=256, I=128), dict(E=6, ranks=2, spare=0, tokens=37, H=136, I=256),
         dict(E=8, ranks=8, spare=1, tokens=30, H=260, I=100, apart=True, dtype=BF16),
         dict(E=8, ranks=4, spare=2, tokens=40, H=200, I=128, masked=True)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_gradients_by_formula_and_by_differences(dev, case, keep):
    s, k, I = Setup(dev, **case), 3, case["I"]
    r, g = s.step(k, keep)
    assert int(r["status"][0]) == 0
    layer, leaves = _plain(s, r["ids"], I)
    out = layer(*leaves)
    dout = s.dout.double().cpu()
    want = torch.autograd.grad((out * dout).sum(), leaves)
    assert _apart(r["out"], out.detach()) < 0.1
    got = (g["x"], g["logits"], g["gate_up"][:, :I], g["gate_up"][:, I:], g["down"])
    for name, a, b in zip(("x", "logits", "gate", "up", "down"), got, want):
        b = torch.where(torch.isfinite(b), b, 0.0)
        assert a.shape == b.shape and _apart(a, b) < 0.1, (name, _apart(a, b))
    # along its own direction each gradient's length is the loss's slope: differences of the plain layer
    for i, a in enumerate(got):
        v = a.double().cpu()
        v = v / v.norm()
        with torch.no_grad():
            eps = 1e-4
            ends = []
            for sign in (1, -1):
                moved = [t.detach() + (sign * eps * v if j == i else 0.0) for j, t in enumerate(leaves)]
                ends.append(float((layer(*moved) * dout).sum()))
        slope = (ends[0] - ends[1]) / (2 * eps)
        assert abs(slope - float(a.double().norm())) < 0.1 * slope
    if case.get("masked"):
        assert (r["out"][3:5] == 0).all() and (g["x"][3:5] == 0).all() and (g["logits"][3:5] == 0).all()
        assert (r["ids"][3:5] == -1).all()


def test_replicas_change_nothing_but_the_order_of_sums(dev):
    with_, without = (Setup(dev, 8, 4, spare, 64, 256, 128) for spare in (2, 0))
    (r, g), (r0, g0) = with_.step(2), without.step(2)
    assert bool((r["plan"].logcnt[0] > 1).any())
    for a, b in ((r["out"], r0["out"]), (g["x"], g0["x"]), (g["logits"], g0["logits"])):
        assert torch.equal(a, b)
    # each sum has at most all pairs' terms, added in another order: both within (pairs + 8) 2^-24 of sum |dy x|
    size = float(max(g0["gate_up"].abs().max(), g0["down"].abs().max()))
    for name in ("gate_up", "down"):
        assert float((g[name] - g0[name]).abs().max()) < 1e-4 * size


def test_fused_layer_against_the_layer_in_steps(dev):
    s = Setup(dev, 8, 4, 1, 64, 256, 128)
    r, _ = s.step(2)
    apart = ep.run_layer(s.x, s.logits, 2, s.layout, s.experts, s.slots)
    assert torch.equal(r["ids"], apart["ids"]) and torch.equal(r["weights"], apart["weights"])
    assert torch.equal(r["src"], apart["src"]) and torch.equal(r["offsets"], apart["offsets"])
    # h rounded with and without its weight, 2.6 % each
    assert _apart(r["out"], apart["out"].double().cpu()) < 0.06


def test_a_step_repeats_bit_for_bit(dev):
    s = Setup(dev, 8, 4, 1, 64, 256, 128)
    (r, g), (r2, g2) = s.step(2), s.step(2)
    assert torch.equal(r["out"], r2["out"]) and all(torch.equal(g[n], g2[n]) for n in g)


def test_refusals(dev):
    s = Setup(dev, 8, 4, 1, 8, 256, 100)
    with pytest.raises(ep.EPBalanceError, match="apart=True"):
        ep.run_layer_train(s.x, s.logits, 2, s.layout, s.experts, s.slots)
    t = Setup(dev, 8, 4, 1, 8, 256, 100, apart=True)
    with pytest.raises(ep.EPBalanceError, match="no gate_up"):
        ep.run_layer(t.x, t.logits, 2, t.layout, t.experts, t.slots)
    with pytest.raises(ep.EPBalanceError, match="same tokens"):
        ep.run_layer_train(t.x, t.logits[:-1], 2, t.layout, t.experts, t.slots)
    with pytest.raises(ep.EPBalanceError, match="keep must be"):
        ep.run_layer_train(t.x, t.logits, 2, t.layout, t.experts, t.slots, keep=torch.float32)
    r = ep.run_layer_train(t.x, t.logits, 2, t.layout, t.experts, t.slots)
    with pytest.raises(ep.EPBalanceError, match="grad_out"):
        ep.run_layer_backward(r, t.dout.float(), t.layout, t.back, t.back_slots)
    with pytest.raises(ep.EPBalanceError, match="must be of hidden"):
        ep.run_layer_backward(r, t.dout, t.layout, ep.ExpertBackwardRows(8, 256, 128, dev), t.back_slots)
    u = Setup(dev, 8, 4, 1, 8, 129, 77, apart=True)
    r = ep.run_layer_train(u.x, u.logits, 2, u.layout, u.experts, u.slots)
    with pytest.raises(ep.EPBalanceError, match="multiple of 4"):
        ep.run_layer_backward(r, u.dout, u.layout, u.back, u.back_slots)


def test_rows_apart_are_the_same_rows_where_halves_are_whole_blocks(dev):
    a, b = Setup(dev, 4, 2, 1, 8, 256, 128), Setup(dev, 4, 2, 1, 8, 256, 128, apart=True)
    assert torch.equal(a.experts.rows, b.experts.rows)
    # transposed matrices hold the same values
    back = S.matrix(a.back.down_t[1], a.back.down_t_scale[1], 256)
    assert torch.equal(back.t(), S.matrix(a.experts.down[1], a.experts.down_scale[1], 128))
    both = S.matrix(a.back.both_t[1], a.back.both_t_scale[1], 256)
    assert torch.equal(both[:, :128].t(), S.matrix(a.experts.gate[1], a.experts.gate_scale[1], 256))
    assert np.prod(a.back.both_t.shape[1:]) == 2 * 128 * 256


def _flat(r, g):
    return [r["out"], r["h"][0].view(torch.uint8), r["kept"][0], g["x"], g["logits"], g["gate_up"], g["down"]]


def test_a_captured_step_replays_as_an_eager_one(dev):
    """The whole step in one graph, replayed over other inputs with eager steps and synchronizations between."""
    s = Setup(dev, 16, 4, 1, 40, 256, 128)
    s.step(2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _flat(*s.step(2))
    gen = torch.Generator(device=dev).manual_seed(5)
    for i in range(4):
        s.x.copy_(torch.randn(s.x.shape, generator=gen, device=dev))
        s.logits.copy_(torch.randn(s.logits.shape, generator=gen, device=dev))
        s.dout.copy_(torch.randn(s.dout.shape, generator=gen, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for a, b in zip(got, _flat(*s.step(2))):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


@pytest.mark.parametrize("tokens,k,spare", [(1, 1, 0), (1, 2, 1), (3, 4, 2)])
def test_few_tokens(dev, tokens, k, spare):
    """A rank's single token, one expert each, no spare slots; the experts that got nothing have gradients of 0."""
    s = Setup(dev, 8, 2, spare, tokens, 128, 256)
    r, g = s.step(k)
    used = torch.zeros(8, dtype=torch.bool, device=dev)
    used[r["ids"].long().flatten()] = True
    for name in ("gate_up", "down"):
        assert torch.isfinite(g[name]).all() and (g[name][~used] == 0).all()
        assert (g[name][used].flatten(1).abs().sum(1) > 0).all()
    assert torch.isfinite(g["x"].float()).all() and torch.isfinite(g["logits"]).all()
    assert (g["x"].float().abs().sum(1) > 0).all()


def test_a_new_workspace_is_no_output(dev, monkeypatch):
    """The workspace that a call makes is apart from all it writes, also where their sizes are alike."""
    from moe_expert_load_layer_amd import layer as module
    seen = []

    class Library:
        def __getattr__(self, name):
            return getattr(ep.lib(), name)

        def ep_grouped_wgrad_mixed(self, p, stream):
            q = p._obj
            seen.append([(q.ws, q.ws_bytes), (q.out, 8 * 64 * 128 * 4), (q.slot_out, 2 * 64 * 128 * 4)])
            return 0

    monkeypatch.setattr(module, "lib", Library)
    lay = ep.Layout.create(8, [4, 4], list(range(8)), [1, 1], device=dev)
    for rows in (64, 256, 1024):        # 256: the workspace is as large as the spare slots' gradients, 1024: as the others'
        x, scale = ep.ep_quant_rows(torch.ones((rows, 128), dtype=BF16, device=dev))
        offsets = torch.full((11,), rows, dtype=torch.int32, device=dev)
        ep.ep_grouped_wgrad_mixed(torch.ones((rows, 64), dtype=BF16, device=dev), x, scale, offsets, layout=lay)
    for ranges in seen:
        for i, (a, n) in enumerate(ranges):
            for b, m in ranges[i + 1:]:
                assert a + n <= b or b + m <= a
    assert len(seen) == 3
