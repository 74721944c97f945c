"""Rows in 8 bits next to the ends of their scale, opened to bf16 by the gated block, its gradient and the weight gradient:
every value under scale bytes from 3 to 246 is taken as it is."""
import pytest
import torch

import swiglu_ref as S
from test_gpu_swiglu import BF16, FP8

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _every_value(dev, code):
    """Row i holds the 8-bit value of code i (of either sign, no NaN) in column i % 128, under one scale byte."""
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8, device=dev)
    q = torch.zeros((len(codes), 128), dtype=torch.uint8, device=dev)
    i = torch.arange(len(codes), device=dev)
    q[i, i % 128] = codes
    scale = torch.full((len(codes), 4), 127, dtype=torch.uint8, device=dev)
    scale[:, 0] = code
    return q.view(FP8), scale, codes.view(FP8).double() * 2.0 ** (code - 127)


@pytest.mark.parametrize("code", [3, 4, 9, 10, 127, 240, 246])
def test_products(dev, code):
    """One value times a power of two that brings it back among the ordinary ones."""
    power = float(2.0 ** max(-100, min(100, 127 - code)))
    x, scale, values = _every_value(dev, code)
    w = ep.ep_quant_blocks(torch.full((1, 160, 128), power, device=dev))
    assert torch.equal(S.matrix(w[0][0], w[1][0], 128), torch.full((160, 128), power, device=dev).double())
    want = (values * power)[:, None].expand(-1, 320)
    _, _, kept, _ = ep.ep_grouped_swiglu(x, scale, *w, *w, keep=BF16)
    assert torch.equal(kept.double(), want)
    # d of the gradient: du = w d a with a = 32, w = 1
    both = torch.full((len(values), 320), 32.0, dtype=BF16, device=dev)
    grad = ep.ep_grouped_swiglu_backward(x, scale, *w, both)[0]
    assert torch.equal(grad[:, 160:].double(), want[:, 160:] * 32)


@pytest.mark.parametrize("code", [3, 4, 9, 10, 127, 240, 246])
@pytest.mark.parametrize("gathered", [False, True])
def test_weight_gradient(dev, code, gathered):
    power = float(2.0 ** max(-100, min(100, 127 - code)))
    x, scale, values = _every_value(dev, code)
    dy = torch.zeros((len(values), 40), dtype=BF16, device=dev)
    i = torch.arange(len(values), device=dev)
    want = torch.zeros((40, 128), dtype=torch.float64, device=dev)
    dy[i, i // 128] = power
    want[i // 128, i % 128] = values * power
    rows = i.to(torch.int32) if gathered else None
    assert torch.equal(ep.ep_grouped_wgrad_mixed(dy, x, scale, x_rows=rows)[0].double(), want)
