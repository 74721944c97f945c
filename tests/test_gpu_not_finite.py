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
