"""Calls on a stream= that is not the current one, with memory that they allocate: while that stream is still busy,
the current one takes and overwrites whatever the allocator hands out."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")

BUSY = 20_000_000       # cycles of a bounded wait, about 10 ms


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _behind(dev, call):
    """call(side stream) behind a wait on it, the current stream overwriting freed memory meanwhile."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out = call(side)
    taken = [torch.full((size,), 255, dtype=torch.uint8, device=dev) for size in (1 << 9, 1 << 13, 1 << 16, 1 << 20)
             for _ in range(24)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert all((t == 255).all() for t in taken)
    return out


def test_layer_for_a_few_tokens(dev):
    E, H, I, T, k = 16, 512, 256, 5, 4
    g = torch.Generator(device=dev).manual_seed(3)
    w = [torch.randn(s, generator=g, device=dev).to(torch.bfloat16) / 10 for s in ((E, I, H), (E, I, H), (E, H, I))]
    x = torch.randn((T, H), generator=g, device=dev).to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device=dev)
    ref = ep.ep_moe_few_tokens(x, logits, k, *w)
    got = _behind(dev, lambda s: ep.ep_moe_few_tokens(x, logits, k, *w, stream=s))
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_eight_bit_inputs_that_only_the_next_call_reads(dev):
    M, N, K = 600, 264, 520
    g = torch.Generator(device=dev).manual_seed(4)
    x, w = torch.randn((M, K), generator=g, device=dev), torch.randn((2, N, K), generator=g, device=dev)
    off = torch.tensor([0, 250, M], dtype=torch.int32, device=dev)

    def product(stream):
        xq, xs = ep.ep_quant_rows(x, stream=stream)
        wq, ws = ep.ep_quant_blocks(w, stream=stream)
        return ep.ep_grouped_matmul(xq, xs, wq, ws, off, stream=stream)

    ref = product(None)
    assert torch.equal(_behind(dev, product), ref)


def test_balancing_path_and_slot_fill(dev):
    lay = ep.Layout.create(16, [2] * 8, list(range(16)), [1] * 8, device=dev)
    g = torch.Generator(device=dev).manual_seed(5)
    ids = (torch.rand((1, 4096), generator=g, device=dev) ** 3 * 16).to(torch.int32)
    rows = torch.randint(0, 255, (16, 1 << 14), generator=g, device=dev, dtype=torch.uint8)

    def path(stream):
        load, ws, status = ep.ep_load_histogram(ids, lay, stream=stream)
        plan = ep.ep_plan_quota(load, lay, status=status, stream=stream)
        slots = torch.zeros((8, 1 << 14), dtype=torch.uint8, device=dev)
        if stream is not None:
            slots.record_stream(stream)
            stream.wait_stream(torch.cuda.current_stream())
        ep.ep_slot_fill(rows, plan.phy2log[0], lay, slots, stream=stream)
        return ep.ep_dispatch_layout(ids, lay, plan.phy_quota, plan.log2phy, plan.logcnt, ws, stream=stream)[1:], slots

    (pos, src), slots = path(None)
    assert (slots != 0).any()
    (pos2, src2), slots2 = _behind(dev, path)
    assert torch.equal(pos, pos2) and torch.equal(src, src2)
    assert torch.equal(slots, slots2)
