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


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[3, 200], [700, 129], [5, 300, 64], [300], [5]])
def test_lists_of_other_tensors(bits, sizes):
    # as after a checkpoint of another shard: numbers of elements and lengths of the scales are those of the new ones
    opt, other = optimizer([5, 300], bits), optimizer(sizes, bits)
    words(opt, [5, 300])
    opt.params, opt.exp_avg, opt.exp_avg_sq = other.params, other.exp_avg, other.exp_avg_sq
    opt.exp_avg_scale, opt.exp_avg_sq_scale = other.exp_avg_scale, other.exp_avg_sq_scale
    w = words(opt, sizes)
    assert w.shape == (len(sizes), 8) and w[:, NUMEL].tolist() == sizes
    assert w[:, PARAM].tolist() == [p.data_ptr() for p in opt.params]
    assert w[:, EXP_AVG].tolist() == [t.data_ptr() for t in opt.exp_avg]
    if bits == 8:
        assert w[:, EXP_AVG_SQ_SCALE].tolist() == [t.data_ptr() for t in opt.exp_avg_sq_scale]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size", [100, 500])
def test_moments_of_another_size_are_refused(bits, size):
    opt = optimizer([5, 300], bits)
    words(opt, [5, 300])
    opt.params[1] = dev(size)
    with pytest.raises(ep.EPBalanceError, match="exp_avg\\[1\\]"):
        words(opt, [5, size])
    if bits == 8:
        other = optimizer([5, size], bits)
        opt.exp_avg, opt.exp_avg_sq = other.exp_avg, other.exp_avg_sq
        with pytest.raises(ep.EPBalanceError, match="exp_avg_scale\\[1\\]"):
            words(opt, [5, size])


def test_values_of_other_tensors(monkeypatch):
    # the values' places are those of the tensors that the lists hold now
    seen = []

    class Library:
        def ep_adamw_values(self, at, n, m, v, stream):
            seen.append((n, v - 0))
            return ep.EP_OK

    monkeypatch.setattr(ep.layer, "lib", Library)
    monkeypatch.setattr(ep.layer, "_stream", lambda s: None)
    opt, other = optimizer([5, 300], 8), optimizer([40, 300, 7], 8)
    opt.params, opt.exp_avg, opt.exp_avg_sq = other.params, other.exp_avg, other.exp_avg_sq
    opt.exp_avg_scale, opt.exp_avg_sq_scale = other.exp_avg_scale, other.exp_avg_sq_scale
    m, v = opt.states()
    assert [t.numel() for t in m] == [t.numel() for t in v] == [40, 300, 7] and seen[0][0] == 3
