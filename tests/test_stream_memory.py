"""Memory that a call allocates is kept until the stream given to it has passed the call: torch's allocator is told of
that stream for every tensor that is not the caller's.  Without a GPU: host tensors pass for device tensors, the
library's entry points are recorded and do nothing."""
import pytest
import torch

import moe_expert_load_layer_amd as ep
from moe_expert_load_layer_amd import layer as M


class Dev(torch.Tensor):
    is_cuda = property(lambda self: True)


def dev(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Dev)


class Stream:
    cuda_stream = 1234


class Library:
    """Records each entry point's integer arguments and answers EP_OK."""

    def __init__(self):
        self.passed = set()

    def __getattr__(self, name):
        def call(*args):
            for a in args:
                a = getattr(a, "value", a)
                if isinstance(a, int):
                    self.passed.add(a)
            return 1 << 10 if name.endswith("bytes") else ep.EP_OK
        return call


@pytest.fixture
def told(monkeypatch):
    """-> (the library, addresses of the tensors that the allocator was told of, addresses that torch.empty gave)"""
    lib, kept, made = Library(), set(), set()
    empty = torch.empty

    def counted(*a, **k):
        t = empty(*a, **k).as_subclass(Dev)
        made.add(t.data_ptr())
        return t

    monkeypatch.setattr(M, "lib", lambda: lib)
    monkeypatch.setattr(ep, "lib", lambda: lib)
    monkeypatch.setattr(torch, "empty", counted)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.add(t.data_ptr()) if s.cuda_stream == 1234
                        else pytest.fail("another stream"))
    return lib, kept, made


def test_workspace_of_the_layer_for_a_few_tokens(told):
    lib, kept, made = told
    bf = torch.bfloat16
    out, ids, w = dev(3, 64, dtype=bf), dev(3, 2, dtype=torch.int32), dev(3, 2)
    ep.ep_moe_few_tokens(dev(3, 64, dtype=bf), dev(3, 4), 2, dev(4, 32, 64, dtype=bf), dev(4, 32, 64, dtype=bf),
                         dev(4, 64, 32, dtype=bf), out=out, ids=ids, weights=w, stream=Stream())
    assert len(made) == 1 and made <= lib.passed and made == kept
