"""The 8-bit grouped product where offsets fall and groups overlap: more tiles than the launch counts on, at K so
short that tiles start afresh and at K where they are chained, for each tile size.  A row of several groups holds one
of their products, every element bit for bit, and nothing outside y is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")

GUARD = 4096


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


# m, n for tiles of 64, 128 and 256
@pytest.mark.parametrize("M,N", [(6400, 64), (3200, 1000), (12288, 1024)])
@pytest.mark.parametrize("K", [100, 384, 512, 640, 700])
@pytest.mark.parametrize("turns", [2, 4])
def test_overlapping_groups(dev, M, N, K, turns):
    print(f"M {M} N {N} K {K} turns {turns}", flush=True)
    g = torch.Generator(device=dev).manual_seed(M + N + K + turns)
    x = torch.randn((M, K), generator=g, device=dev)
    G = 2 * turns - 1                                     # every other group is empty, the rest own all rows
    w = torch.randn((G, N, K), generator=g, device=dev)
    xq, xs = ep.ep_quant_rows(x)
    wq, ws = ep.ep_quant_blocks(w)
    off = torch.tensor([0, M] * turns, dtype=torch.int32, device=dev)
    buf = torch.full((M * N + 2 * GUARD,), 7.0, dtype=torch.bfloat16, device=dev)
    y = buf[GUARD:GUARD + M * N].view(M, N)
    ep.ep_grouped_matmul(xq, xs, wq, ws, off, y=y)
    left = torch.ones((M, N), dtype=torch.bool, device=dev)
    for e in range(0, G, 2):
        left &= y != ep.ep_grouped_matmul(xq, xs, wq[e:e + 1], ws[e:e + 1])
    assert not left.any()
    assert (buf[:GUARD] == 7).all() and (buf[GUARD + M * N:] == 7).all()


def test_overlapping_weight_gradients(dev):
    # each group sums its own rows, also where they are another's too
    M, N, K = 700, 72, 264
    g = torch.Generator(device=dev).manual_seed(1)
    dy = torch.randn((M, N), generator=g, device=dev).to(torch.bfloat16)
    x = torch.randn((M, K), generator=g, device=dev).to(torch.bfloat16)
    off = torch.tensor([0, M, 0, M, 300, 200, M], dtype=torch.int32, device=dev)
    out = ep.ep_grouped_wgrad(dy, x, off)
    whole = ep.ep_grouped_wgrad(dy, x)[0]
    assert torch.equal(out[0], whole) and torch.equal(out[2], whole)
    assert (out[1] == 0).all() and (out[3] == 0).all() and (out[4] == 0).all()
    assert torch.equal(out[5], ep.ep_grouped_wgrad(dy[200:].contiguous(), x[200:].contiguous())[0])
