"""run_layer refuses x and logits of different tokens before it enqueues anything, without a GPU: host tensors pass for
device tensors."""
import pytest
import torch

import moe_expert_load_layer_amd as ep


class Dev(torch.Tensor):
    is_cuda = property(lambda self: True)


def dev(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Dev)


@pytest.mark.parametrize("tokens", [5, 7])
def test_run_layer_refuses(monkeypatch, tokens):
    def enqueue(*a):
        raise AssertionError("the library is called")

    monkeypatch.setattr(ep, "lib", enqueue)
    monkeypatch.setattr(ep.layer, "lib", enqueue)
    monkeypatch.setattr(ep.layer, "_stream", lambda s: None)
    lay = ep.Layout(4, 2, 6, 2, 2, dev(64, dtype=torch.int32), ep._CLayout())
    rows, slots = ep.ExpertRows(4, 128, 128, "cpu"), ep.ExpertRows(2, 128, 128, "cpu")
    with pytest.raises(ep.EPBalanceError, match="same tokens"):
        ep.run_layer(dev(6, 128, dtype=torch.bfloat16), dev(tokens, 4), 2, lay, rows, slots)
