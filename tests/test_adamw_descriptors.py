"""The descriptors that AdamW passes to the library after its lists were changed, without a GPU: host tensors pass for
device tensors."""
import pytest
import torch

import moe_expert_load_layer_amd as ep

PARAM, GRAD, EXP_AVG, EXP_AVG_SQ, EXP_AVG_SCALE, EXP_AVG_SQ_SCALE, COPY, NUMEL = range(8)


class Dev(torch.Tensor):
    is_cuda = property(lambda self: True)


def dev(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Dev)


def optimizer(sizes, bits=32, copies=False):
    opt = ep.AdamW([dev(n) for n in sizes], bits=bits,
                   copies=[dev(n, dtype=torch.bfloat16) for n in sizes] if copies else None)
    for tensors in (opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale):
        if tensors is not None:
            tensors[:] = [t.as_subclass(Dev) for t in tensors]
    return opt


def words(opt, sizes):
    opt._tensors([dev(n) for n in sizes])
    return opt._words


@pytest.mark.parametrize("bits", [32, 8])
def test_no_copies_any_more(bits):
    opt = optimizer([5, 300], bits, copies=True)
    assert (words(opt, [5, 300])[:, COPY] != 0).all()
    opt.copies = None
    assert (words(opt, [5, 300])[:, COPY] == 0).all()
