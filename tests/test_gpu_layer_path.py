"""The gate, the balancer and the experts' products as one layer: the example runs, its prefill agrees with the plain
64-bit layer on 8-bit weights, its folded gradient with the plain gradient, and its step lowers the loss."""
import os
import sys

import numpy as np
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _plain(x, ids, w, gate_up, down, inter):
    """The layer with 8-bit weights and inputs, rounded where the path rounds."""
    T, H = x.shape
    xq, _ = R.quant_rows(x)
    out = np.zeros((T, H))
    gu, dn = [R.quant_blocks(m)[0] for m in gate_up], [R.quant_blocks(m)[0] for m in down]
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if e >= 0:
                u = gu[e] @ xq[t]
                h, _ = R.quant_rows((R.silu(u[:inter]) * u[inter:])[None])
                out[t] += w[t, j] * (dn[e] @ h[0])
    return out


def test_example(dev):
    import moe_layer as M
    r = M.main(dev)
    pre, T = r["pre"], 24
    w = ep.ExpertRows(M.EXPERTS, M.HIDDEN, M.INTER, dev)
    assert int(pre["status"][0]) == 0 and bool((pre["plan"].logcnt[0] > 1).any())    # replicas are in use
    # prefill: an 8-bit rounding of h may fall the other way after the bf16 rounding of its inputs (2^-9 of a value
    # against steps of 2^-3): in the 2-norm that and the bf16 roundings stay below 3 %
    rng = np.random.default_rng(0)
    some = rng.choice(r["x"].shape[0], T, replace=False)
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    gate_up = torch.randn((M.EXPERTS, 2 * M.INTER, M.HIDDEN), generator=g, device=dev) * M.HIDDEN ** -0.5
    down = torch.randn((M.EXPERTS, M.HIDDEN, M.INTER), generator=g, device=dev) * M.INTER ** -0.5
    ids, wts = pre["ids"].cpu().numpy(), pre["weights"].double().cpu().numpy()
    ref = _plain(r["x"].double().cpu().numpy()[some], ids[some], wts[some], gate_up.double().cpu().numpy(),
                 down.double().cpu().numpy(), M.INTER)
    got = pre["out"].double().cpu().numpy()[some]
    assert np.linalg.norm(got - ref) < 0.03 * np.linalg.norm(ref)
    # decode differs by the 8-bit rounding of x and h, about 2.6 % each
    assert r["apart"] < 0.06
    # every replica's share is in the native gradient: as if each expert had taken all its pairs
    up = pre["up"].float()
    h = (torch.nn.functional.silu(up[:, :M.INTER]) * up[:, M.INTER:]).to(torch.bfloat16).double()
    src = pre["src"].long()
    dy = (r["target"][src // M.TOP_K] * pre["weights"].view(-1)[src][:, None]).to(torch.bfloat16).double()
    of = pre["ids"].view(-1)[src]
    for e in range(M.EXPERTS):
        at = of == e
        want, size = dy[at].t() @ h[at], dy[at].abs().t() @ h[at].abs()
        assert ((r["native"][e].double() - want).abs() <= (int(at.sum()) + 16) * 2.0 ** -24 * size).all()
    assert r["after"] < r["before"]
    assert w.rows.shape == (M.EXPERTS, w.rows.shape[1]) and w.rows.shape[1] % 16 == 0


def test_run_layer_with_padded_tokens_and_no_spares(dev):
    lay = ep.Layout.create(4, [2, 2], [0, 1, 2, 3], [0, 0], device=dev)
    rows = ep.ExpertRows(4, 128, 128, dev).load(torch.randn((4, 256, 128), device=dev) / 11,
                                                torch.randn((4, 128, 128), device=dev) / 11)
    none = ep.ExpertRows(0, 128, 128, dev)
    x = torch.randn((20, 128), device=dev).to(torch.bfloat16)
    logits = torch.randn((20, 4), device=dev)
    logits[7:9] = -float("inf")
    r = ep.run_layer(x, logits, 2, lay, rows, none)
    assert (r["out"][7:9] == 0).all() and (r["out"][:7] != 0).any()
    keep = [t for t in range(20) if t not in (7, 8)]
    alone = ep.run_layer(x[keep], logits[keep], 2, lay, rows, none)
    assert torch.equal(r["out"][keep], alone["out"])
