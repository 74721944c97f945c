"""The gate and its gradient against the plain 64-bit form.

IDs are exact: the scores are the inputs plus one fp32 addition.  Weights: exp's argument is a difference
rounded once (2^-24 of at most 32 in these inputs), exp within 2 ulp, k + 2 roundings in sum and quotient:
(32 + 2 + k + 2) 2^-24 < 4e-6 relative.  Gradients: three more roundings of values below sum |w g|."""
import numpy as np
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _logits(rng, T, E, dtype):
    x = torch.from_numpy(rng.normal(0, 2, (T, E)).astype(np.float32)).clamp(-8, 8)
    return x.to(dtype)


def _check(dev, logits, k, bias=None, groups=1, topk_groups=1, scale=1.0):
    ids, w = ep.ep_gate_topk(logits.to(dev), k, bias=None if bias is None else torch.from_numpy(bias).to(dev),
                             num_groups=groups, topk_groups=topk_groups, scale=scale)
    rid, rw = R.gate(logits.float().numpy(), bias, k, groups, topk_groups, scale)
    assert np.array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=4e-6, atol=1e-37)
    return ids, w, rid, rw


@pytest.mark.parametrize("T,E,k,groups,topk_groups", [
    (1, 1, 1, 1, 1), (1, 8, 8, 1, 1), (3, 12, 2, 1, 1), (17, 128, 8, 1, 1), (64, 256, 8, 8, 4), (5, 160, 8, 5, 3),
    (33, 384, 8, 1, 1), (7, 385, 16, 1, 1), (9, 1000, 6, 8, 2), (2, 1024, 16, 16, 16), (31, 96, 3, 4, 1),
    (16, 130, 8, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_matches(dev, T, E, k, groups, topk_groups, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    bias = rng.normal(0, 0.5, E).astype(np.float32) if E % 2 == 0 else None
    _check(dev, _logits(rng, T, E, dtype), k, bias, groups, topk_groups, scale=1.0 if T % 2 else 2.5)


def test_gate_ties_go_to_the_lowest_expert(dev):
    logits = torch.zeros((4, 96))
    logits[1, 40:60] = 1.0
    logits[2] = torch.where(torch.arange(96) % 2 == 0, -0.0, 0.0)       # -0 equals 0
    logits[3] = torch.full((96,), torch.finfo(torch.float32).min)        # the lowest finite value is a score
    ids, w, _, _ = _check(dev, logits, 4)
    assert ids[0].tolist() == [0, 1, 2, 3] and ids[1].tolist() == [40, 41, 42, 43]
    assert ids[2].tolist() == [0, 1, 2, 3] and w[3].tolist() == [0.25] * 4
    _check(dev, logits, 4, groups=4, topk_groups=2)


@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (4, 2)])
def test_gate_switched_off_experts_and_padded_tokens(dev, groups, topk_groups):
    rng = np.random.default_rng(5)
    logits = _logits(rng, 9, 32, torch.float32)
    logits[0] = -np.inf                       # nothing left: -1 and weight 0
    logits[1, 1:] = -np.inf                   # one expert left
    logits[2, ::2] = -np.inf
    logits[3, 5] = np.nan                     # NaN is never chosen
    logits[4] = np.nan
    logits[5, 7] = np.inf                     # takes all the weight
    logits[6, 3] = logits[6, 30] = np.inf     # or an equal share of it
    ids, w, _, _ = _check(dev, logits, 4, None, groups, topk_groups)
    assert ids[0].tolist() == [-1] * 4 and w[0].tolist() == [0.0] * 4
    assert ids[1].tolist() == [0, -1, -1, -1] and w[1].tolist() == [1.0, 0, 0, 0]
    assert ids[4].tolist() == [-1] * 4
    assert ids[5, 0].item() == 7 and w[5, 0].item() == 1.0


def test_gate_strided_and_unaligned_logits(dev):
    rng = np.random.default_rng(6)
    wide = _logits(rng, 21, 200, torch.float32).to(dev)
    for view in (wide[:, 3:131], wide[:, 8:136], wide[::2, :64]):
        ids, w = ep.ep_gate_topk(view, 8)
        rid, rw = R.gate(view.cpu().numpy(), None, 8, 1, 1)
        assert np.array_equal(ids.cpu().numpy(), rid)
        np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=4e-6)


@pytest.mark.parametrize("T,E,k,scale", [(1, 8, 2, 1.0), (19, 128, 8, 2.5), (64, 385, 16, 1.0), (16, 256, 8, 0.0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_backward(dev, T, E, k, scale, dtype):
    rng = np.random.default_rng(E)
    logits = _logits(rng, T, E, torch.float32)
    logits[0, 1:] = -np.inf
    ids, w = ep.ep_gate_topk(logits.to(dev), k, scale=scale)
    grad = rng.normal(0, 1, (T, k)).astype(np.float32)
    got = ep.ep_gate_topk_backward(ids, w, torch.from_numpy(grad).to(dev), E, scale=scale, dtype=dtype)
    rid, rw = R.gate(logits.numpy(), None, k, 1, 1, scale)
    ref = R.gate_backward(rid, rw, grad.astype(np.float64), E, scale)
    size = np.abs(rw * grad).sum(axis=1, keepdims=True) + np.abs(rw) .max() * np.abs(grad).max()
    tol = size * 1e-5 + (np.abs(ref) * 2.0 ** -8 if dtype == torch.bfloat16 else 0)
    assert (np.abs(got.float().cpu().numpy() - ref) <= tol + 1e-37).all()


def test_gate_backward_matches_differences(dev):
    # d(sum_j g_j w_j) / dl by central differences of the 64-bit weights
    rng = np.random.default_rng(8)
    T, E, k, scale, h = 3, 24, 4, 1.5, 1e-5
    logits = rng.normal(0, 1, (T, E)).astype(np.float32)
    ids, w = ep.ep_gate_topk(torch.from_numpy(logits).to(dev), k, scale=scale)
    g = rng.normal(0, 1, (T, k)).astype(np.float32)
    got = ep.ep_gate_topk_backward(ids, w, torch.from_numpy(g).to(dev), E, scale=scale).cpu().numpy()
    rid = ids.cpu().numpy()

    def value(l, t):
        z = l[rid[t]]
        e = np.exp(z - z.max())
        return (g[t] * scale * e / e.sum()).sum()

    for t in range(T):
        for e in range(E):
            a, b = logits[t].astype(np.float64), logits[t].astype(np.float64)
            a[e] += h
            b[e] -= h
            assert abs((value(a, t) - value(b, t)) / (2 * h) - got[t, e]) < 1e-5


def test_gate_no_tokens_and_given_outputs(dev):
    ids, w = ep.ep_gate_topk(torch.empty((0, 16), device=dev), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert ep.ep_gate_topk_backward(ids, w, w, 16).shape == (0, 16)
    logits = torch.randn((5, 16), device=dev)
    ids, w = torch.empty((5, 4), dtype=torch.int32, device=dev), torch.empty((5, 4), device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = ep.ep_gate_topk(logits, 4, ids=ids, weights=w, stream=side)
    side.synchronize()
    assert a is ids and b is w
    assert torch.equal(ids.long(), torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :4])


def test_gate_ids_feed_the_histogram(dev):
    lay = ep.Layout.create(16, [2] * 8, list(range(16)), [1] * 8, device=dev)
    logits = torch.randn((64, 16), device=dev)
    logits[60:] = -np.inf                      # padded tokens
    ids, _ = ep.ep_gate_topk(logits, 2)
    load, _, status = ep.ep_load_histogram(ids.view(1, -1), lay)
    assert int(status[0]) == 0 and int(load.sum()) == 120
    assert torch.equal(load[0].long(), torch.bincount(ids[ids >= 0].long(), minlength=16))
