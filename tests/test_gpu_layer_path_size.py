"""run_layer and the slots' weight gradients over a whole layout: 256 experts on 64 ranks with 32 spare slots, 7168 x
2048, group-limited routing.  Every part is compared with its plain form in 64 bits on the inputs that it had: each
pair's products with its native expert's weights, whichever slot served it.

Bounds are those of the parts' own tests: an 8-bit product 7 2^-13 of the sum of magnitudes and half a bf16 ulp, an
8-bit rounding of h half a step, the combine (k + 1) 2^-24, a weight gradient (m + 8) 2^-24."""
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _rows(q, s):
    kb = q.shape[-1] // 128
    return q.double() * torch.exp2(s[..., :kb].double() - 127).repeat_interleave(128, dim=-1)


def _matrix(q, s):
    unit = torch.exp2(s.double() - 127).repeat_interleave(128, dim=0)[:q.shape[0]].repeat_interleave(128, dim=1)
    return (q.double() * unit).T.contiguous()


def _close(y, a, w):
    ref, mag = a @ w, a.abs() @ w.abs()
    assert ((y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 7 * 2.0 ** -13 * mag + 1e-30).all()


def test_layer_over_a_whole_layout(dev):
    wl = W.get("deepseek_v3").scaled(tokens_per_rank=16)
    lay = ep.Layout.from_workload(wl, device=dev)
    E, k, T, (H, I) = wl.num_experts, wl.top_k, wl.num_ranks * wl.tokens_per_rank, wl.expert_shape[1:]
    g = torch.Generator(device=dev).manual_seed(1)
    experts, slots = ep.ExpertRows(E, H, I, dev), ep.ExpertRows(lay.num_spare, H, I, dev)
    gate_up = torch.randn((E, 2 * I, H), generator=g, device=dev, dtype=torch.bfloat16) * H ** -0.5
    down = torch.randn((E, H, I), generator=g, device=dev, dtype=torch.bfloat16) * I ** -0.5
    experts.load(gate_up, down)
    del gate_up, down
    x = torch.randn((T, H), generator=g, device=dev).to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device=dev) + 2 * torch.randn(E, generator=g, device=dev)
    logits[5] = -float("inf")                                  # a padded token
    r = ep.run_layer(x, logits, k, lay, experts, slots, num_groups=8, topk_groups=4)
    assert int(r["status"][0]) == 0 and bool((r["plan"].logcnt[0] > 1).any())
    ids, pos, src, M = r["ids"].view(-1).long(), r["pos"].long(), r["src"].long(), int(r["offsets"][-1])
    assert M == (T - 1) * k and torch.equal(pos[src[:M]], torch.arange(M, device=dev))

    xv, hv = _rows(*ep.ep_quant_rows(x)), _rows(*r["h"])
    up = r["up"].double()
    a = up[:, :I] / (1 + torch.exp(-up[:, :I])) * up[:, I:]
    unit = torch.exp2(r["h"][1][:, :I // 128].double() - 127).repeat_interleave(128, dim=1)
    assert ((hv[:M] - a[:M]).abs() <= (a[:M].abs() * 2.0 ** -4 + unit[:M] * 2.0 ** -10) * (1 + 1e-5)).all()
    for e in range(E):
        at = pos[(ids == e).nonzero()[:, 0]]
        if len(at):
            _close(r["up"][at], xv[src[at] // k], _matrix(experts.gate_up[e], experts.gate_up_scale[e]))
            _close(r["y"][at], hv[at], _matrix(experts.down[e], experts.down_scale[e]))
    assert (r["y"][M:] == 0).all()
    y, w = r["y"].double(), r["weights"].double()
    here = (pos >= 0).view(T, k, 1)
    terms = torch.where(here, w[:, :, None] * y[pos.clamp(min=0)].view(T, k, H), 0.0)
    ref, mag = terms.sum(dim=1), terms.abs().sum(dim=1)
    assert ((r["out"].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (k + 1) * 2.0 ** -24 * mag).all()
    assert (r["out"][5] == 0).all()

    dy, h = torch.randn((T * k, H), generator=g, device=dev).to(torch.bfloat16), hv.to(torch.bfloat16)
    native, spare = ep.ep_grouped_wgrad(dy, h, r["offsets"], layout=lay)
    first, home = [int(v) for v in r["offsets"]], r["plan"].phy2log[0].tolist()
    at, spares, seen = 0, 0, set()
    for rank in range(wl.num_ranks):
        for j in range(wl.native_count[rank] + wl.spare_count[rank]):
            i, n = first[at], first[at + 1] - first[at]
            got = native[home[at]] if j < wl.native_count[rank] else spare[spares]
            if j >= wl.native_count[rank]:
                spares += 1
            if at % 5 == 0 or j >= wl.native_count[rank]:
                d, b = dy[i:i + n].double().T.contiguous(), h[i:i + n].double()
                assert ((got.double() - d @ b).abs() <= (n + 8) * 2.0 ** -24 * (d.abs() @ b.abs())).all(), at
                seen.add(j >= wl.native_count[rank] and n > 0)
            at += 1
    assert at == lay.num_phys and spares == lay.num_spare and seen == {False, True}
