"""An infinity in one row of the gated block or its gradient, beside rows whose largest value is exactly 448 times a
power of two, the most that a block's scale leaves room for: the others keep their scales, and so does the infinite row's
own finite part."""
import pytest
import torch

import swiglu_ref as S
from test_gpu_swiglu import BF16, FP8

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")

INF = float("inf")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _matrix(values, dev):
    """[N][128] with `values` in column 0, in 8 bits; exact for values of 4 bits."""
    w = torch.zeros((1, len(values), 128), device=dev)
    w[0, :, 0] = values
    q, s = ep.ep_quant_blocks(w)
    assert torch.equal(S.matrix(q[0], s[0], 128), w[0].double())
    return q, s


def _ones(M, dev):
    x = torch.zeros((M, 128), dtype=BF16, device=dev)
    x[:, 0] = 1
    return ep.ep_quant_rows(x)


def _inputs(dev, large, unit=2.0 ** -5):
    """Values of 4 bits up to `large`, and down to where a scale twice as large as `unit` would drop their last bits."""
    values = torch.tensor([1.0, 1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875], device=dev).repeat(16)
    values = values * 2.0 ** -(torch.arange(128, device=dev) // 8 % 14)
    values = (values / unit).to(FP8).float() * unit
    values[7] = large
    return values


# the tiles of 64, 128 and 256 rows, with sums of either kind
@pytest.mark.parametrize("M,blocks", [(40, 1), (200, 1), (17000, 2)])
@pytest.mark.parametrize("sums8", [False, True], ids=["fp32", "8bit"])
@pytest.mark.parametrize("keep", [None, BF16, FP8], ids=["none", "bf16", "fp8"])
def test_forward(dev, M, blocks, sums8, keep):
    values = _inputs(dev, 14.0).repeat(blocks)
    gate, up = _matrix(torch.full_like(values, 32.0), dev), _matrix(values, dev)   # sigmoid(32) is 1 in fp32
    x, weights = _ones(M, dev), torch.ones(M, device=dev)
    clean = ep.ep_grouped_swiglu(*x, *gate, *up, weights=weights, keep=keep, sums8=sums8)
    want = S.values(*clean[:2])
    assert torch.equal(want, (values * 32).double().expand(M, -1)) and (clean[1][:, :blocks] == 127).all()
    bad = torch.zeros(M, dtype=torch.bool, device=dev)
    bad[[5, M // 2, M - 1]] = True
    weights[bad] = INF
    h, hs, kept, ks = ep.ep_grouped_swiglu(*x, *gate, *up, weights=weights, keep=keep, sums8=sums8)
    assert torch.equal(h.view(torch.uint8)[~bad], clean[0].view(torch.uint8)[~bad])
    assert torch.equal(hs[~bad], clean[1][~bad]) and torch.isnan(h.float()[bad]).all()
    for a, b in ((kept, clean[2]), (ks, clean[3])):
        assert a is b or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("M,blocks", [(40, 1), (200, 1), (70000, 4)])
@pytest.mark.parametrize("sums8", [False, True], ids=["fp32", "8bit"])
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_backward(dev, M, blocks, sums8, keep):
    """du = 32 w d with g = 32, and dg = w u d: both blocks have a largest value of 448."""
    values = _inputs(dev, 14.0).repeat(blocks)
    wide = len(values)
    down = _matrix(values, dev)
    both = torch.full((M, 2 * wide), 32.0, dtype=BF16, device=dev)
    kept, ks = ep.ep_quant_rows(both) if keep is FP8 else (both, None)
    dy, weights = _ones(M, dev), torch.ones(M, device=dev)
    run = lambda: ep.ep_grouped_swiglu_backward(*dy, *down, kept, ks, weights=weights, sums8=sums8)  # noqa: E731
    clean = run()
    assert torch.equal(S.values(*clean[1:3]), (values * 32).double().repeat(2).expand(M, -1))
    assert (clean[2][:, :2 * blocks] == 127).all()
    bad = torch.zeros(M, dtype=torch.bool, device=dev)
    bad[[5, M // 2, M - 1]] = True
    weights[bad] = INF
    grad, q, qs, dw = run()
    assert torch.equal(q.view(torch.uint8)[~bad], clean[1].view(torch.uint8)[~bad])
    assert torch.equal(qs[~bad], clean[2][~bad]) and torch.equal(grad[~bad], clean[0][~bad])
    assert torch.isnan(q.float()[bad]).all() and torch.isinf(grad.float()[bad]).all() and torch.equal(dw, clean[3])


@pytest.mark.parametrize("sums8", [False, True], ids=["fp32", "8bit"])
@pytest.mark.parametrize("M", [40, 200])
def test_the_finite_part_of_an_infinite_row(dev, sums8, M):
    """A row with one infinite value has the smallest scale that holds the others: at 448 and just above it."""
    for large, code in ((14.0, 127), (13.0, 127), (15.0, 128)):
        values = _inputs(dev, large, 1.0)
        values[3] = 448.0                       # x 448 x 2^120 overflows
        gate, up = _matrix(torch.full_like(values, 32.0), dev), _matrix(values, dev)
        weights = torch.ones(M, device=dev)
        row = M // 3
        for power in (0, 115):
            weights[:] = 2.0 ** power
            h, hs, _, _ = ep.ep_grouped_swiglu(*_ones(M, dev), *gate, *up, weights=weights, sums8=sums8)
            infinite = values.double() * 32 * 2.0 ** power >= 2.0 ** 128
            assert torch.equal(torch.isnan(h.float()[row]), infinite) and infinite.any() == (power == 115)
            if power:
                assert (hs[row, 0] == code + power).all()
                assert torch.equal(S.values(h, hs)[row][~infinite], (values.double() * 32 * 2.0 ** power)[~infinite])


@pytest.mark.parametrize("sums8", [False, True], ids=["fp32", "8bit"])
@pytest.mark.parametrize("M,blocks", [(40, 1), (200, 1), (70000, 4)])
@pytest.mark.parametrize("keep", [BF16, FP8], ids=["bf16", "fp8"])
def test_the_finite_part_of_infinite_gradients(dev, sums8, M, blocks, keep):
    for large, code in ((14.0, 127), (13.0, 127), (15.0, 128)):
        values = _inputs(dev, large, 1.0)
        values[3] = 448.0
        values = values.repeat(blocks)
        both = torch.full((M, 2 * len(values)), 32.0, dtype=BF16, device=dev)
        kept, ks = ep.ep_quant_rows(both) if keep is FP8 else (both, None)
        weights = torch.ones(M, device=dev)
        row = M // 3
        weights[row] = 2.0 ** 115
        _, q, qs, _ = ep.ep_grouped_swiglu_backward(*_ones(M, dev), *_matrix(values, dev), kept, ks, weights=weights,
                                                    sums8=sums8)
        want = values.double().repeat(2) * 32 * 2.0 ** 115
        infinite = want >= 2.0 ** 128
        assert infinite.any() and torch.equal(torch.isnan(q.float()[row]), infinite)
        assert (qs[row, :2 * blocks] == code + 115).all()
        assert torch.equal(S.values(q[row:row + 1], qs[row:row + 1])[0][~infinite], want[~infinite])
        assert (qs[row + 1, :2 * blocks] == 132).all() and not torch.isnan(q.float()[row + 1]).any()
