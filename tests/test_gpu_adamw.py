"""AdamW against its formula in 64 bits, and its 8-bit states against an fp32 replica of the defined rounding.

32-bit: a step's moments carry 4 roundings (both coefficients' own among them) of values that the same recurrence
over |g| bounds, its parameter about 8 of values below |p| + lr: over S steps 8 S 2^-24 (|p| + lr) bounds the
parameter, and 4 S 2^-24 the moments relative to the recurrence over |g| (m's terms may cancel).
8 bits: every operation up to the code is a single IEEE fp32 operation, so the codes are equal bit for bit."""
import numpy as np
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")

HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _grads(rng, sizes, dtype, step):
    return [torch.from_numpy((rng.normal(0, 1e-3, n) * np.exp(rng.normal(0, 2, n))).astype(np.float32)).to(dtype)
            for n in sizes]


@pytest.mark.parametrize("sizes", [[1], [7, 128, 129], [2048, 2047, 2049, 1, 0, 5], [300000]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("copy", [False, True])
def test_adamw_32(dev, sizes, dtype, copy):
    rng = np.random.default_rng(len(sizes))
    p0 = [rng.normal(0, 0.05, n).astype(np.float32) for n in sizes]
    params = [torch.from_numpy(p).to(dev) for p in p0]
    copies = [torch.full((n,), 7.0, dtype=torch.bfloat16, device=dev) for n in sizes] if copy else None
    opt = ep.AdamW(params, copies=copies, **HP)
    ref = [(p.astype(np.float64), np.zeros(len(p)), np.zeros(len(p))) for p in p0]
    size = [np.zeros(len(p)) for p in p0]
    S = 5
    for t in range(1, S + 1):
        g = _grads(rng, sizes, dtype, t)
        opt.step([x.to(dev) for x in g], grad_scale=0.5)
        ref = [R.adamw(*r, x.double().numpy() * 0.5, t, *[HP[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay")])
               for r, x in zip(ref, g)]
        size = [HP["beta1"] * a + (1 - HP["beta1"]) * np.abs(x.double().numpy() * 0.5) for a, x in zip(size, g)]
    m, v = opt.states()
    u = 2.0 ** -24
    for i, (p, rm, rv) in enumerate(ref):
        assert (np.abs(params[i].cpu().numpy() - p) <= 8 * S * u * (np.abs(p) + HP["lr"] * S)).all()
        assert (np.abs(m[i].cpu().numpy() - rm) <= 4 * S * u * size[i]).all()
        assert (np.abs(v[i].cpu().numpy() - rv) <= 4 * S * u * rv).all()
        if copy:
            assert torch.equal(copies[i], params[i].to(torch.bfloat16))


def _mix(h):
    h = (h * np.uint32(0x9E3779B9)).astype(np.uint32)
    h ^= h >> np.uint32(15)
    h = (h * np.uint32(0x6A09E667)).astype(np.uint32)
    h ^= h >> np.uint32(13)
    h = (h * np.uint32(0xBB67AE85)).astype(np.uint32)
    return h ^ (h >> np.uint32(16))


def _codes(x, noise, low, signed):
    n = len(x)
    t = np.zeros(-(-n // 128) * 128, np.float32)
    t[:n] = np.abs(x)
    amax = t.reshape(-1, 128).max(axis=1)
    # 2^(c - 127) is the smallest power of two with amax <= 1.875 of it
    e = np.array([1 if a == 0 else int(np.clip(127 + np.ceil(np.log2(float(a) / 1.875) - 1e-12), 1, 253)) for a in amax])
    inv = np.exp2((127.0 - e)).astype(np.float32)
    bits = (t.reshape(-1, 128) * inv[:, None]).astype(np.float32).reshape(-1)[:n].view(np.uint32)
    c = ((bits + noise) >> np.uint32(20)).astype(np.int64) - low
    if signed:
        return np.clip(c, 0, 127) | np.where(x < 0, 128, 0), e
    return np.where(x > 0, np.clip(c, 1, 255), 0), e


def _values(q, e, low, signed):
    mag = q & 127 if signed else q
    x = np.where(mag > 0, ((mag + low).astype(np.uint32) << np.uint32(20)).view(np.float32), np.float32(0))
    x = (x * np.exp2(e.astype(np.float64) - 127).astype(np.float32).repeat(128)[:len(q)]).astype(np.float32)
    return np.where(q > 127, -x, x) if signed else x


@pytest.mark.parametrize("sizes", [[1], [127, 128, 129, 1000], [5003, 4097]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_adamw_8_codes_are_the_defined_ones(dev, sizes, dtype):
    rng = np.random.default_rng(11)
    params = [torch.from_numpy(rng.normal(0, 0.05, n).astype(np.float32)).to(dev) for n in sizes]
    seed = 0xFFFFFFF0
    opt = ep.AdamW(params, bits=8, seed=seed, **HP)
    f = np.float32
    state = [[np.zeros(n, f), np.zeros(n, f)] for n in sizes]
    for t in range(1, 5):
        g = _grads(rng, sizes, dtype, t)
        opt.step([x.to(dev) for x in g])
        vals = opt.states()
        for i, n in enumerate(sizes):
            x = g[i].float().numpy()
            m = state[i][0] * f(HP["beta1"]) + x * f(1 - HP["beta1"])
            v = state[i][1] * f(HP["beta2"]) + (x * x) * f(1 - HP["beta2"])
            with np.errstate(over="ignore"):
                h = _mix((np.arange(n, dtype=np.uint64) + seed + t * 0x9E3779B9 + i * 0x6A09E667).astype(np.uint32))
                rm = (h * np.uint32(0x9E3779B9)).astype(np.uint32) >> np.uint32(12)
            qm, em = _codes(m, rm, 896, True)
            qv, ev = _codes(v, h & np.uint32(0xFFFFF), 768, False)
            assert np.array_equal(opt.exp_avg_scale[i].cpu().numpy(), em)
            assert np.array_equal(opt.exp_avg_sq_scale[i].cpu().numpy(), ev)
            assert np.array_equal(opt.exp_avg[i].cpu().numpy(), qm)
            assert np.array_equal(opt.exp_avg_sq[i].cpu().numpy(), qv)
            state[i] = [_values(qm, em, 896, True), _values(qv, ev, 768, False)]
            assert np.array_equal(vals[0][i].cpu().numpy(), state[i][0])
            assert np.array_equal(vals[1][i].cpu().numpy(), state[i][1])
            assert (qv[x != 0] > 0).all()          # a second moment is never lost


def test_adamw_8_follows_the_moments(dev):
    # constant gradients: m tends to g and v to g^2; a code is 1/8 of its power of two wide, and the random
    # rounding walks around the mean: over 16384 elements the mean's deviation is far below one code
    n, S = 16384, 400
    g = torch.full((n,), 0.02, device=dev)
    p = torch.zeros(n, device=dev)
    opt = ep.AdamW([p], bits=8, lr=1e-3, beta1=0.9, beta2=0.99, weight_decay=0.0, seed=3)
    for _ in range(S):
        opt.step([g])
    m, v = opt.states()
    assert abs(m[0].double().mean().item() / 0.02 - 1) < 0.02
    assert abs(v[0].double().mean().item() / 4e-4 - 1) < 0.03
    assert abs(-p.double().mean().item() / (S * 1e-3) - 1) < 0.1


def test_adamw_many_tensors_views_and_streams(dev):
    # more tensors than one launch's descriptors hold; parts of one buffer at odd offsets; a side stream
    rng = np.random.default_rng(4)
    for bits in (32, 8):
        buf = torch.from_numpy(rng.normal(0, 1, 120 * 70).astype(np.float32)).to(dev)
        gbuf = torch.from_numpy(rng.normal(0, 1, 120 * 70).astype(np.float32)).to(dev)
        at = [i * 70 + i % 4 for i in range(120)]
        params, grads = [buf[a:a + 61] for a in at], [gbuf[a:a + 61] for a in at]
        one = [torch.zeros(61, device=dev).copy_(x) for x in params]
        before = buf.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a, b = ep.AdamW(params, bits=bits, seed=9), ep.AdamW(one, bits=bits, seed=9)
        torch.cuda.synchronize()
        for _ in range(3):
            a.step(grads, stream=side)
            b.step(grads)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(params, one))
        touched = torch.zeros(len(buf), dtype=torch.bool, device=dev)
        for i in at:
            touched[i:i + 61] = True
        assert torch.equal(buf[~touched], before[~touched]) and not torch.equal(buf[touched], before[touched])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_infinite_gradients_show(dev, bits):
    p = torch.ones(300, device=dev)
    g = torch.ones(300, device=dev)
    g[5], g[200] = float("inf"), float("nan")
    opt = ep.AdamW([p], bits=bits, **HP)
    opt.step([g])
    assert torch.isnan(p[5]) and torch.isnan(p[200])
    assert int(torch.isnan(p).sum()) == 2


def test_adamw_repeats_bit_for_bit(dev):
    outs = []
    for _ in range(2):
        g = torch.Generator(device=dev)
        g.manual_seed(1)
        p = torch.randn(100003, generator=g, device=dev)
        opt = ep.AdamW([p], bits=8, seed=5, **HP)
        for _ in range(4):
            opt.step([torch.randn(100003, generator=g, device=dev)])
        outs.append((p, opt.exp_avg[0], opt.exp_avg_sq[0]))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
