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

    monkeypatch.setattr(torch, "empty_like", lambda t: counted(t.shape, dtype=t.dtype))
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


def _calls():
    bf, i32, u8, fp8 = torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn
    eight = lambda *s: dev(*s, dtype=u8).view(fp8)                       # noqa: E731
    lay = ep.Layout(4, 2, 6, 2, 2, dev(64, dtype=i32), ep._CLayout())
    off, s = dev(3, dtype=i32), Stream()
    opt = ep.AdamW([dev(200)], bits=8)
    for moments in (opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale):
        moments[:] = [m.as_subclass(Dev) for m in moments]
    return dict(
        gate=(2, lambda: ep.ep_gate_topk(dev(5, 8), 2, stream=s)),
        gate_backward=(1, lambda: ep.ep_gate_topk_backward(dev(5, 2, dtype=i32), dev(5, 2), dev(5, 2), 8, stream=s)),
        quant_rows=(2, lambda: ep.ep_quant_rows(dev(5, 200), stream=s)),
        swiglu=(2, lambda: ep.ep_swiglu_quant(dev(5, 200, dtype=bf), stream=s)),
        quant_blocks=(2, lambda: ep.ep_quant_blocks(dev(2, 30, 200), stream=s)),
        matmul=(1, lambda: ep.ep_grouped_matmul(eight(5, 128), dev(5, 4, dtype=u8), eight(2, 30, 128),
                                                dev(2, 1, 1, dtype=u8), off, stream=s)),
        wgrad=(1, lambda: ep.ep_grouped_wgrad(dev(5, 30, dtype=bf), dev(5, 20, dtype=bf), off, stream=s)),
        wgrad_slots=(2, lambda: ep.ep_grouped_wgrad(dev(5, 30, dtype=bf), dev(5, 20, dtype=bf), dev(7, dtype=i32),
                                                    layout=lay, stream=s)),
        combine=(1, lambda: ep.ep_moe_combine(dev(5, 16, dtype=bf), dev(3, 2, dtype=i32), dev(3, 2), stream=s)),
        few_tokens=(4, lambda: ep.ep_moe_few_tokens(dev(3, 64, dtype=bf), dev(3, 4), 2, dev(4, 32, 64, dtype=bf),
                                                    dev(4, 32, 64, dtype=bf), dev(4, 64, 32, dtype=bf), stream=s)),
        adamw_values=(1, lambda: opt.states(stream=s)))


@pytest.mark.parametrize("name", ["gate", "gate_backward", "quant_rows", "swiglu", "quant_blocks", "matmul", "wgrad",
                                  "wgrad_slots", "combine", "few_tokens", "adamw_values"])
def test_outputs_of_the_layer_s_operators(told, name):
    # a caller may drop them at once, as an 8-bit input that only the next call reads
    lib, kept, made = told
    count, call = _calls()[name]
    made.clear()
    call()
    assert len(made) == count and made == kept


@pytest.mark.parametrize("name", ["histogram", "plan", "reroute", "dispatch", "stats", "slot_fill", "path"])
def test_memory_of_the_balancing_path(told, name):
    lib, kept, made = told
    i32 = torch.int32
    lay, s = ep.Layout(4, 2, 6, 2, 2, dev(64, dtype=i32), ep._CLayout()), Stream()
    ids, load, ws = dev(1, 20, dtype=i32), dev(1, 4, dtype=i32), dev(4096, dtype=torch.uint8)
    plan = (dev(1, 6, dtype=i32), dev(1, 4, 2, dtype=i32), dev(1, 4, dtype=i32))
    count, call = dict(
        histogram=(3, lambda: ep.ep_load_histogram(ids, lay, stream=s)),
        plan=(5, lambda: ep.ep_plan_quota(load, lay, stream=s)),
        reroute=(1, lambda: ep.ep_reroute(ids, lay, *plan, ws, stream=s)),
        dispatch=(3, lambda: ep.ep_dispatch_layout(ids, lay, *plan, ws, stream=s)),
        stats=(3, lambda: ep.ep_balance_stats(load, plan[0], lay, stream=s)),
        slot_fill=(1, lambda: ep.ep_slot_fill(dev(4, 32), dev(6, dtype=i32), lay, dev(2, 32), stream=s)),
        path=(12, lambda: ep.run_path(ids, lay, stream=s)))[name]
    call()
    assert len(made) == count and made == kept
