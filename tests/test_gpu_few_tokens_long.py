"""The layer for a few tokens where a workgroup of either kernel goes through more than 512 windows of 8-bit weights,
so that it fetches scale bytes more than once: wide rows for gate and up, many pairs on few shares for down.

16 experts that all 64 tokens choose, 50040 x 1160: 32 entries of up to 32 pairs by 37 row tiles, 1184 items of 391
windows for at most 768 workgroups; 64 entries of up to 16 pairs by 10 windows in one share.

Bounds as for the other sizes: h carries the fp32 sums of gate and up, here 1564 additions of 32 products, whose
roundings are 2^-24 of partial sums that stay near the final one's size and add at random: 40 2^-24, below 2^-18
of what a sum of that size is; two bf16 (2^-17); in all 2^-13 of the terms' magnitudes, and the output's bf16."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _values(q, s, cols):
    unit = torch.exp2(s.double() - 127).repeat_interleave(128, dim=0)[:q.shape[0]].repeat_interleave(128, dim=1)
    return (q.double() * unit)[:, :cols]


def test_many_windows(dev):
    T, E, k, H, I = 64, 16, 16, 50040, 1160
    g = torch.Generator(device=dev).manual_seed(1)

    def weights(n, c):
        w = torch.randn((E, n, c), generator=g, device=dev, dtype=torch.bfloat16) * c ** -0.5
        # blocks of different sizes, so that a scale byte of another window shows
        w *= torch.exp2(torch.randint(-2, 3, (E, 1, -(-c // 128)), generator=g, device=dev).float()
                        ).repeat_interleave(128, dim=2)[..., :c].to(torch.bfloat16)
        return ep.ep_quant_blocks(w)

    (gq, gs), (uq, us), (dq, ds) = weights(I, H), weights(I, H), weights(H, I)
    x = torch.randn((T, H), generator=g, device=dev).to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device=dev)
    out, ids, w = ep.ep_moe_few_tokens(x, logits, k, gq, uq, dq, gs, us, ds)
    dense = torch.zeros((T, E), dtype=torch.float64, device=dev).scatter_(1, ids.long(), w.double())
    assert torch.equal(ids.long().sort(dim=1).values, torch.arange(E, device=dev).expand(T, E))
    ref, mag = torch.zeros((T, H), dtype=torch.float64, device=dev), torch.zeros((T, H), dtype=torch.float64, device=dev)
    for e in range(E):
        a = x.double() @ _values(gq[e], gs[e], H).T.contiguous()
        h = a / (1 + torch.exp(-a)) * (x.double() @ _values(uq[e], us[e], H).T.contiguous())
        d = _values(dq[e], ds[e], I).T.contiguous()
        ref += dense[:, e:e + 1] * (h @ d)
        mag += dense[:, e:e + 1].abs() * (h.abs() @ d.abs())
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * mag).all()
