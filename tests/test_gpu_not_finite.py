"""Infinities and NaN in blocks of 128 that share a scale byte stay where they are: the block's other values are those
that they are without them, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_moments_of_a_block(dev, value, dtype):
    # elements 5 and 300 are lost in the second step; in the other run they have gradient 0
    g = torch.Generator(device=dev).manual_seed(1)
    p0, grads = torch.randn(400, generator=g, device=dev), torch.randn((4, 400), generator=g, device=dev) * 1e-3
    lost = torch.zeros(400, dtype=torch.bool, device=dev)
    lost[5] = lost[300] = True
    runs = []
    for bad in (value, 0.0):
        p = p0.clone()
        opt = ep.AdamW([p], bits=8, seed=7, lr=1e-2)
        for t in range(4):
            x = torch.where(lost, bad if t == 1 else 0.0, grads[t]).to(dtype)
            opt.step([x])
        m, v = opt.states()
        runs.append([p, m[0], v[0], opt.exp_avg_scale[0], opt.exp_avg_sq_scale[0]])
    (p, m, v, ms, vs), (rp, rm, rv, rms, rvs) = runs
    assert torch.equal(ms, rms) and torch.equal(vs, rvs)
    assert torch.isnan(p[lost]).all()
    for a, b in ((p, rp), (m, rm), (v, rv)):
        assert torch.equal(a[~lost], b[~lost])


def _apart(dev, dtype, bad):
    """A matrix [200][300] and the same with `bad` in three places."""
    g = torch.Generator(device=dev).manual_seed(2)
    w = torch.randn((200, 300), generator=g, device=dev).to(dtype)
    lost = torch.zeros((200, 300), dtype=torch.bool, device=dev)
    lost[5, 7] = lost[130, 131] = lost[199, 299] = True
    return torch.where(lost, torch.zeros_like(w), w), torch.where(lost, torch.full_like(w, bad), w), lost


def _only_lost_differ(a, b, lost):
    """8-bit values and scale bytes, the second with NaN where `lost`."""
    (q, s), (qb, sb) = a, b
    assert torch.equal(s, sb)
    q, qb = q.view(torch.uint8)[..., :lost.shape[-1]], qb.view(torch.uint8)[..., :lost.shape[-1]]
    assert torch.equal(q[~lost], qb[~lost]) and ((qb[lost] & 127) == 127).all()


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_eight_bit_blocks(dev, bad, dtype):
    w, wb, lost = _apart(dev, dtype, bad)
    _only_lost_differ(ep.ep_quant_rows(w), ep.ep_quant_rows(wb), lost)
    _only_lost_differ(ep.ep_quant_blocks(w[None]), ep.ep_quant_blocks(wb[None]), lost[None])
    _only_lost_differ(ep.ep_quant_blocks(w[None], transpose=True), ep.ep_quant_blocks(wb[None], transpose=True),
                      lost.t()[None])


@pytest.mark.parametrize("bad", [INF, NAN])
def test_eight_bit_blocks_of_silu(dev, bad):
    u, ub, lost = _apart(dev, torch.bfloat16, bad)
    gate = torch.full_like(u, 1.5)
    _only_lost_differ(ep.ep_swiglu_quant(torch.cat([gate, u], dim=1)), ep.ep_swiglu_quant(torch.cat([gate, ub], dim=1)),
                      lost)


def test_product_with_an_infinite_weight(dev):
    # one infinite weight makes its own column of y infinite or NaN, and no other one smaller
    w, wb, lost = _apart(dev, torch.bfloat16, INF)
    g = torch.Generator(device=dev).manual_seed(3)
    xq, xs = ep.ep_quant_rows(torch.randn((40, 300), generator=g, device=dev))
    y, yb = (ep.ep_grouped_matmul(xq, xs, *ep.ep_quant_blocks(m[None])) for m in (w, wb))
    column = lost.any(dim=1)
    assert torch.isnan(yb[:, column]).all() and torch.equal(y[:, ~column], yb[:, ~column])


@pytest.mark.parametrize("scale", [1e-39, -3e-39, 2.0 ** -128, 1e-30])
def test_gate_gradient_with_the_smallest_scales(dev, scale):
    # 1 / scale is not finite below 2^-128; w, w g and their sum are whole multiples of 2^-149, rounded once or twice
    # each: (k + 3) 2^-149 for the mean's numerator, which dividing by the scale and multiplying by w <= |scale| keeps
    T, E, k = 9, 16, 4
    g = torch.Generator(device=dev).manual_seed(6)
    logits, grad = torch.randn((T, E), generator=g, device=dev), torch.randn((T, k), generator=g, device=dev)
    ids, w = ep.ep_gate_topk(logits, k, scale=scale)
    got = ep.ep_gate_topk_backward(ids, w, grad, E, scale=scale)
    assert torch.isfinite(got).all()
    s, a = float(torch.tensor(scale, dtype=torch.float32)), w.double()
    d = a * (grad.double() - (a * grad.double()).sum(dim=1, keepdim=True) / s)
    ref = torch.zeros((T, E), dtype=torch.float64, device=dev).scatter_(1, ids.long(), d)
    size = a.abs() * (grad.double().abs() + (a * grad.double()).abs().sum(dim=1, keepdim=True) / abs(s))
    bound = torch.zeros_like(ref).scatter_(1, ids.long(), (k + 6) * 2.0 ** -24 * size) + (k + 6) * 2.0 ** -149
    assert ((got.double() - ref).abs() <= bound).all()
