"""A mixture-of-experts layer with the balancer inside it, as a program would use it:

  prefill  the gate, the balanced path and the experts' 8-bit products over the physical slots, replicas included;
  decode   the same layer for a few tokens in one call;
  train    one step on the down matrices: the weight gradient of every physical slot, replicas folded into their
           native expert, AdamW with 8-bit states, new 8-bit weights.

Run `python examples/moe_layer.py` on an MI355X; `main` returns what it printed.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_load_layer_amd as ep  # noqa: E402

EXPERTS, RANKS, TOP_K, HIDDEN, INTER, TOKENS = 16, 8, 4, 512, 256, 96   # TOKENS: of each rank


def relative(a: torch.Tensor, b: torch.Tensor) -> float:
    return float((a.double() - b.double()).norm() / b.double().norm())


def main(device="cuda:0", seed=0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device=device)     # noqa: E731

    # 2 experts and 1 spare slot on each rank; fp32 parameters, 8-bit weights for the products
    layout = ep.Layout.create(EXPERTS, [2] * RANKS, list(range(EXPERTS)), [1] * RANKS, device=device)
    gate_up = randn(EXPERTS, 2 * INTER, HIDDEN) * HIDDEN ** -0.5
    down = randn(EXPERTS, HIDDEN, INTER) * INTER ** -0.5
    experts = ep.ExpertRows(EXPERTS, HIDDEN, INTER, device).load(gate_up, down)
    slots = ep.ExpertRows(layout.num_spare, HIDDEN, INTER, device)

    x = randn(RANKS * TOKENS, HIDDEN).to(torch.bfloat16)
    logits = randn(RANKS * TOKENS, EXPERTS) + 3 * torch.rand(EXPERTS, generator=g, device=device)
    pre = ep.run_layer(x, logits, TOP_K, layout, experts, slots)
    loads = ep.ep_balance_stats(ep.ep_load_histogram(pre["ids"].view(1, -1), layout)[0], pre["plan"].phy_quota,
                                layout)[1]
    print(f"prefill: {x.shape[0]} tokens, imbalance {float(loads[0, 0]):.2f} -> {float(loads[0, 1]):.2f}")

    # decode: the first tokens again, weights as they are stored, inputs in bf16
    few = 5
    gate, up = experts.gate_up[:, :INTER], experts.gate_up[:, INTER:]
    gate_scale, up_scale = experts.gate_up_scale[:, :INTER // 128], experts.gate_up_scale[:, INTER // 128:]
    dec, ids, _ = ep.ep_moe_few_tokens(x[:few], logits[:few], TOP_K, gate, up, experts.down, gate_scale, up_scale,
                                       experts.down_scale)
    assert torch.equal(ids, pre["ids"][:few])
    apart = relative(dec, pre["out"][:few])
    print(f"decode:  {few} tokens, {apart:.3f} from prefill, which rounds its inputs to 8 bits")

    # train: L = sum(out * target); the gradient of each pair's output row is its weight times the target
    target = randn(RANKS * TOKENS, HIDDEN)
    src = pre["src"].long().clamp(min=0)
    taken = (pre["src"] >= 0).float()[:, None]
    dy = (target[src // TOP_K] * pre["weights"].view(-1)[src][:, None] * taken).to(torch.bfloat16)
    a, b = pre["up"].float().chunk(2, dim=1)
    h = (torch.nn.functional.silu(a) * b * taken).to(torch.bfloat16)
    native, spare = ep.ep_grouped_wgrad(dy, h, pre["offsets"], layout=layout)
    ep.ep_replica_grad_reduce(native.view(EXPERTS, -1), spare.view(layout.num_spare, -1), pre["plan"].log2phy[0],
                              pre["plan"].logcnt[0], layout)
    before = float((pre["out"].double() * target.double()).sum())
    opt = ep.AdamW([down], bits=8, lr=2e-3, weight_decay=0.0, seed=seed)
    opt.step([native])
    experts.load(gate_up, down)
    after = float((ep.run_layer(x, logits, TOP_K, layout, experts, slots)["out"].double() * target.double()).sum())
    print(f"train:   loss {before:.1f} -> {after:.1f} after one step")
    return dict(layout=layout, x=x, logits=logits, gate_up=gate_up, target=target, pre=pre, few=dec, apart=apart,
                native=native, before=before, after=after)


if __name__ == "__main__":
    main()
