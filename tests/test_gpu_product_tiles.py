"""The 8-bit grouped product where a workgroup takes many tiles one after the other: every tile size, ragged and
empty groups, scales over several chunks, widths that leave part tiles, gathered rows with holes, rows past the
last group, and the same call again.

The plain form multiplies the rounded values (their bytes and scales as ep_quant_rows and ep_quant_blocks gave
them) in 64 bits.  Bounds as for one tile: each 8 products lose at most 7 2^-13 of their sum of magnitudes, the
bf16 output rounds by 2^-9 of itself; in the 2-norm 2^-9 and a quarter of it."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _rows(q, s):
    """float64 values of 8-bit rows [M][kb * 128] with a scale byte for each 128."""
    kb = q.shape[-1] // 128
    unit = torch.exp2(s[..., :kb].double() - 127).repeat_interleave(128, dim=-1)
    return q.double() * unit


def _matrix(q, s):
    unit = torch.exp2(s.double() - 127).repeat_interleave(128, dim=0)[:q.shape[0]].repeat_interleave(128, dim=1)
    return q.double() * unit


def _sizes(rng, M, G, spread):
    """G ragged sizes that leave some rows over; every fifth group is empty."""
    a = rng.random(G) ** spread
    a[2::5] = 0
    return np.floor(a / a.sum() * (M - M // 50)).astype(np.int64)


@pytest.mark.parametrize("M,N,K,G,spread,gather", [
    (8192, 2304, 1500, 5, 1, False), (8192, 2304, 4300, 3, 1, True), (8100, 2301, 700, 4, 2, True),
    (8192, 2304, 1500, 64, 1, True), (4096, 2304, 4300, 40, 2, False), (4000, 2301, 900, 30, 1, False),
    (2048, 2304, 1500, 128, 1, False), (2048, 2304, 4300, 100, 2, True), (2000, 2301, 1000, 90, 1, True)])
def test_many_tiles(dev, M, N, K, G, spread, gather):
    rng = np.random.default_rng(M + N + K + G)
    g = torch.Generator(device=dev).manual_seed(K)
    T = M // 3 if gather else M
    x = torch.randn((T, K), generator=g, device=dev)
    x *= torch.exp(torch.randn((T, 1), generator=g, device=dev))
    w = torch.randn((G, N, K), generator=g, device=dev, dtype=torch.bfloat16)
    xq, xs = ep.ep_quant_rows(x)
    wq, ws = ep.ep_quant_blocks(w)
    sizes = _sizes(rng, M, G, spread)
    ends = np.concatenate([[0], np.cumsum(sizes)])
    off = torch.tensor(ends, dtype=torch.int32, device=dev)
    rows = rng.integers(-T // 20, 2 * T + 3, M) if gather else np.arange(M)   # some negative, some too large
    at = np.where((rows < 0) | (rows // 2 >= T), -1, rows // 2) if gather else rows
    r = torch.tensor(rows, dtype=torch.int32, device=dev) if gather else None
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev)
    ep.ep_grouped_matmul(xq, xs, wq, ws, off, rows=r, rows_div=2 if gather else 1, y=y)
    first = y.clone()
    xv, at = _rows(xq, xs), torch.tensor(at, device=dev)
    missed, square, total = 0.0, 0.0, 0.0
    for e in range(G):
        i, j = int(ends[e]), int(ends[e + 1])
        if i == j:
            continue
        a = torch.where((at[i:j] >= 0)[:, None], xv[at[i:j].clamp(min=0)], 0.0)
        wv = _matrix(wq[e], ws[e])
        ref, mag = a @ wv.T.contiguous(), a.abs() @ wv.abs().T.contiguous()
        d = (y[i:j].double() - ref).abs()
        assert (d <= 2.0 ** -8 * ref.abs() + 7 * 2.0 ** -13 * mag + 1e-30).all(), e
        square, total = square + float((d * d).sum()), total + float((ref * ref).sum())
    assert square ** 0.5 <= 1.25 * 2.0 ** -9 * total ** 0.5
    assert (y[int(ends[-1]):] == 0).all() and int(ends[-1]) < M
    y.fill_(3.0)
    ep.ep_grouped_matmul(xq, xs, wq, ws, off, rows=r, rows_div=2 if gather else 1, y=y)
    assert torch.equal(y, first)


@pytest.mark.parametrize("N,K,sizes", [(1160, 2568, (170, 0, 130)), (2048, 4096, (64, 33)), (3000, 1031, (200,))])
def test_wgrad_many_tiles(dev, N, K, sizes):
    # exact products of bf16, fp32 additions: (m + 8) 2^-24 of the sum of magnitudes
    M = sum(sizes)
    g = torch.Generator(device=dev).manual_seed(N)
    dy = torch.randn((M, N), generator=g, device=dev).to(torch.bfloat16)
    x = torch.randn((M, K), generator=g, device=dev).to(torch.bfloat16)
    ends = np.concatenate([[0], np.cumsum(sizes)])
    off = torch.tensor(ends, dtype=torch.int32, device=dev)
    got = ep.ep_grouped_wgrad(dy, x, off, out=torch.full((len(sizes), N, K), 7.0, device=dev))
    for e, m in enumerate(sizes):
        i, j = int(ends[e]), int(ends[e + 1])
        a, b = dy[i:j].double().T.contiguous(), x[i:j].double()
        assert ((got[e].double() - a @ b).abs() <= (m + 8) * 2.0 ** -24 * (a.abs() @ b.abs())).all(), e
