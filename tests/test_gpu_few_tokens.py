"""The layer for a few tokens against the plain 64-bit form.

IDs exact, weights as the gate's.  Output: with S the sum of |w down h| over all terms, h carries the fp32 sums of
gate and up (relative to their own terms' magnitudes; these inputs cancel by less than 2^5) and two bf16 (2^-17),
the down sums another few 2^-24 S times the additions: 2^-13 S in all; the output half a bf16 ulp, 2^-9 |out|."""
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


def _weights(rng, E, N, K, fp8, dev):
    w = torch.from_numpy((rng.normal(0, 1, (E, N, K)) / np.sqrt(K)).astype(np.float32)).to(torch.bfloat16)
    if not fp8:
        return w.to(dev), None, w.double().numpy()
    q, s = ep.ep_quant_blocks(w.to(dev))
    return q, s, np.stack([R.quant_blocks(w[e].double().numpy())[0] for e in range(E)])


def _layer(rng, dev, T, E, k, H, I, fp8, groups=1, topk_groups=1, masked=False, bias=None, ldtype=torch.float32,
           sharp=0.0):
    x = torch.from_numpy(rng.normal(0, 1, (T, H)).astype(np.float32)).to(torch.bfloat16)
    l = rng.normal(0, 1.5, (T, E))
    l[:, :max(1, k)] += sharp
    logits = torch.from_numpy(l.astype(np.float32)).to(ldtype)
    if masked:
        logits[:, ::5] = -np.inf
        logits[::3] = -np.inf
    (g, gs, gv), (u, us, uv) = _weights(rng, E, I, H, fp8, dev), _weights(rng, E, I, H, fp8, dev)
    d, ds, dv = _weights(rng, E, H, I, fp8, dev)
    out, ids, w = ep.ep_moe_few_tokens(x.to(dev), logits.to(dev), k, g, u, d, gs, us, ds,
                                       bias=None if bias is None else torch.from_numpy(bias).to(dev),
                                       num_groups=groups, topk_groups=topk_groups)
    rid, rw = R.gate(logits.float().numpy(), bias, k, groups, topk_groups)
    assert np.array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=4e-6, atol=1e-37)
    ref, mag = R.layer(x.double().numpy(), rid, rw, gv, uv, dv)
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * mag).all()
    return got, rid


@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 8, 8), (1, 8, 2, 64, 32), (2, 12, 3, 72, 40), (5, 16, 8, 200, 136), (16, 128, 8, 256, 128),
    (33, 8, 4, 264, 72), (64, 4, 3, 128, 64), (64, 130, 8, 136, 264), (7, 385, 6, 520, 16), (3, 1000, 16, 64, 8)])
@pytest.mark.parametrize("fp8", [False, True])
def test_layer_matches(dev, T, E, k, H, I, fp8):
    _layer(np.random.default_rng(T * E + H), dev, T, E, k, H, I, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_groups_bias_masks(dev, fp8):
    rng = np.random.default_rng(2)
    got, ids = _layer(rng, dev, 12, 32, 4, 136, 72, fp8, groups=8, topk_groups=3, masked=True,
                      bias=rng.normal(0, 0.5, 32).astype(np.float32), ldtype=torch.bfloat16)
    assert (ids[::3] == -1).all() and (got[::3] == 0).all()
    got, ids = _layer(rng, dev, 3, 16, 2, 64, 64, fp8, masked=True)     # few or no experts left
    assert (got[0] == 0).all()


@pytest.mark.parametrize("T", [16, 17, 32, 33, 64])
def test_layer_all_tokens_on_the_same_experts(dev, T):
    # every expert's token list is full: one, two and four column tiles
    _layer(np.random.default_rng(T), dev, T, 40, 3, 192, 80, False, sharp=40.0)


def test_layer_packed_rows_strides_and_workspace(dev):
    # the three matrices of an expert as parts of one row, x and logits as views, given outputs
    rng = np.random.default_rng(7)
    E, H, I, T, k = 6, 72, 40, 5, 2
    rows = torch.from_numpy(rng.normal(0, 0.2, (E, 3 * H * I)).astype(np.float32)).to(torch.bfloat16).to(dev)
    g, u = rows[:, :H * I].unflatten(1, (I, H)), rows[:, H * I:2 * H * I].unflatten(1, (I, H))
    d = rows[:, 2 * H * I:].unflatten(1, (H, I))
    x = torch.from_numpy(rng.normal(0, 1, (T, 2 * H)).astype(np.float32)).to(torch.bfloat16).to(dev)[:, H:]
    logits = torch.from_numpy(rng.normal(0, 1, (T, E + 3)).astype(np.float32)).to(dev)[:, 1:E + 1]
    a = ep.ep_moe_few_tokens(x, logits, k, g, u, d)
    ws = torch.full((ep.ep_few_tokens_workspace_bytes(T, k, H, I),), 255, dtype=torch.uint8, device=dev)
    outs = (torch.full((T, H), 9.0, dtype=torch.bfloat16, device=dev),
            torch.full((T, k), 9, dtype=torch.int32, device=dev), torch.full((T, k), 9.0, device=dev))
    b = ep.ep_moe_few_tokens(x.contiguous(), logits.contiguous(), k, g.contiguous(), u.contiguous(), d.contiguous(),
                             out=outs[0], ids=outs[1], weights=outs[2], ws=ws)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert ep.ep_moe_few_tokens(x[:0], logits[:0], k, g, u, d)[0].shape == (0, H)


def test_layer_values_do_not_leak(dev):
    # NaN in an expert that nobody chooses, or in one token, stays there
    rng = np.random.default_rng(8)
    E, H, I, T = 8, 200, 72, 4
    x = torch.randn((T, H), device=dev).to(torch.bfloat16)
    logits = torch.zeros((T, E), device=dev)
    logits[:, :2] = 5
    w = [torch.from_numpy(rng.normal(0, 0.1, s).astype(np.float32)).to(torch.bfloat16).to(dev)
         for s in ((E, I, H), (E, I, H), (E, H, I))]
    a = ep.ep_moe_few_tokens(x, logits, 2, *w)[0]
    for t in w:
        t[2:] = float("nan")
    x2 = x.clone()
    x2[3] = float("inf")
    b = ep.ep_moe_few_tokens(x2, logits, 2, *w)[0]
    assert torch.equal(a[:3], b[:3]) and torch.isnan(b[3]).any()


def test_layer_in_a_graph_and_on_a_side_stream(dev):
    # replays read the inputs' new values; eager calls run between them
    E, H, I, T, k = 16, 256, 128, 3, 4
    w = [torch.randn(s, device=dev).to(torch.bfloat16) / 10 for s in ((E, I, H), (E, I, H), (E, H, I))]
    x, logits = torch.randn((T, H), device=dev).to(torch.bfloat16), torch.randn((T, E), device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = ep.ep_moe_few_tokens(x, logits, k, *w)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(eager, ep.ep_moe_few_tokens(x, logits, k, *w)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = ep.ep_moe_few_tokens(x, logits, k, *w)
    for _ in range(4):
        x.copy_(torch.randn((T, H), device=dev))
        logits.copy_(torch.randn((T, E), device=dev))
        graph.replay()
        ref = ep.ep_moe_few_tokens(x, logits, k, *w)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, ref))
