"""The 8-bit grouped product, its rounding, the weight gradient and the steps between, against the plain
64-bit forms.

Rounding to 8 bits is exact arithmetic (powers of two, one rounding to nearest): values and scale bytes are
equal bit for bit.  Product: the matrix instruction aligns each 8 products to their largest and drops what lies
below 2^-13 of it (measured: beside 2^16, 2^3 is kept and 2^2 lost among the same 8, and kept elsewhere), so 7
dropped rests below 2^-13 max <= 2^-13 sum |x w| a group bound its error, 7 2^-13 sum |x w| in all; bf16 output
adds half an ulp, 2^-9 |y|.  The rests are far smaller as a rule: in the 2-norm the bf16 rounding (at most 2^-9)
and a quarter of it for them have to do.  Weight gradient: products of bf16 are exact in fp32, additions rounded:
(m + 8) 2^-24 sum |dy x| at the most."""
import numpy as np
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

ep = pytest.importorskip("moe_expert_load_layer_amd")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _x(rng, M, K, dtype=torch.bfloat16):
    a = rng.normal(0, 1, (M, K)) * np.exp(rng.normal(0, 1, (M, 1)))
    a[:, rng.random(K) < 0.02] *= 30
    return torch.from_numpy(a.astype(np.float32)).to(dtype)


def _bytes(q):
    return q.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (5, 129), (17, 200), (64, 1536), (33, 1000), (2, 4096)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quant_rows(dev, M, K, dtype):
    rng = np.random.default_rng(M * K)
    x = _x(rng, M, K, dtype)
    if M > 2:
        x[1] = 0
        x[2] = 1e-38
    q, s = ep.ep_quant_rows(x.to(dev))
    val, e = R.quant_rows(x.double().numpy())
    kb = -(-K // 128)
    got = R.FP8[_bytes(q)] * np.exp2(s.cpu().numpy()[:, :kb].astype(float) - 127).repeat(128, axis=1)
    assert np.array_equal(s.cpu().numpy()[:, :kb], e + 127)
    assert (s.cpu().numpy()[:, kb:] == 127).all() and s.shape[1] % 4 == 0
    assert np.array_equal(got[:, :K], val) and (got[:, K:] == 0).all()


def test_quant_rows_strided_unaligned_and_not_finite(dev):
    rng = np.random.default_rng(2)
    wide = _x(rng, 12, 400).to(dev)
    for view in (wide[:, 3:300], wide[:, 8:264], wide[::3, :256]):
        q, s = ep.ep_quant_rows(view)
        val, _ = R.quant_rows(view.double().cpu().numpy())
        K = view.shape[1]
        got = R.FP8[_bytes(q)] * np.exp2(s.cpu().numpy()[:, :-(-K // 128)].astype(float) - 127).repeat(128, axis=1)
        assert np.array_equal(got[:, :K], val)
    x = torch.ones((2, 256), dtype=torch.bfloat16, device=dev)
    x[0, 3], x[0, 200], x[1, 130] = float("inf"), float("nan"), float("-inf")
    q, _ = ep.ep_quant_rows(x)
    bad = np.isnan(R.FP8[_bytes(q)])
    assert bad[0].nonzero()[0].tolist() == [3, 200] and bad[1].nonzero()[0].tolist() == [130]


@pytest.mark.parametrize("G,N,K", [(1, 1, 1), (2, 128, 128), (3, 130, 257), (2, 64, 300), (1, 384, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quant_blocks_and_transposed(dev, G, N, K, dtype):
    rng = np.random.default_rng(N * K)
    w = torch.stack([_x(rng, N, K, dtype) for _ in range(G)])
    q, s = ep.ep_quant_blocks(w.to(dev))
    qt, st = ep.ep_quant_blocks(w.to(dev), transpose=True)
    assert q.shape == (G, N, -(-K // 128) * 128) and qt.shape == (G, K, -(-N // 128) * 128)
    for g in range(G):
        val, e = R.quant_blocks(w[g].double().numpy())
        sg, tg = s[g].cpu().numpy(), st[g].cpu().numpy()
        assert np.array_equal(sg, e + 127) and np.array_equal(tg, e.T + 127)
        unit = np.exp2(sg.astype(float) - 127).repeat(128, axis=0)[:N].repeat(128, axis=1)
        got = R.FP8[_bytes(q[g])] * unit
        assert np.array_equal(got[:, :K], val) and (got[:, K:] == 0).all()
        tv = R.FP8[_bytes(qt[g])] * np.exp2(tg.astype(float) - 127).repeat(128, axis=0)[:K].repeat(128, axis=1)
        assert np.array_equal(tv[:, :N], val.T) and (tv[:, N:] == 0).all()


def test_quant_blocks_of_a_packed_row(dev):
    # one matrix inside packed expert rows: groups further apart than their size
    rows = torch.randn((4, 3 * 64 * 96), device=dev)
    part = rows[:, 64 * 96:2 * 64 * 96].unflatten(1, (64, 96))
    a, sa = ep.ep_quant_blocks(part)
    b, sb = ep.ep_quant_blocks(part.contiguous())
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(sa, sb)


def _offsets(sizes, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=dev)


def _product(rng, dev, M, N, K, sizes, rows=None, div=1):
    """The kernel's output and the plain one with the bound of their distance."""
    G = len(sizes)
    T = M if rows is None else max(1, -(-M // div))
    x = _x(rng, T, K).to(dev)
    w = torch.from_numpy((rng.normal(0, 1, (G, N, K)) / np.sqrt(K)).astype(np.float32)).to(dev)
    xq, xs = ep.ep_quant_rows(x)
    wq, ws = ep.ep_quant_blocks(w)
    off = _offsets(sizes, dev)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev)
    r = None if rows is None else torch.from_numpy(rows.astype(np.int32)).to(dev)
    ep.ep_grouped_matmul(xq, xs, wq, ws, off, rows=r, rows_div=div, y=y)
    xv, _ = R.quant_rows(x.double().cpu().numpy())
    ref, mag = np.zeros((M, N)), np.zeros((M, N))
    at = np.arange(M) if rows is None else np.where(rows < 0, -1, rows // div)
    for g in range(G):
        i, j = int(sum(sizes[:g])), int(sum(sizes[:g + 1]))
        wv, _ = R.quant_blocks(w[g].double().cpu().numpy())
        a = np.where((at[i:j] >= 0)[:, None], xv[np.clip(at[i:j], 0, T - 1)], 0.0)
        ref[i:j], mag[i:j] = a @ wv.T, np.abs(a) @ np.abs(wv).T
    return y.double().cpu().numpy(), ref, mag


def _close(y, ref, mag):
    assert (np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 7 * 2.0 ** -13 * mag + 1e-30).all()
    assert np.linalg.norm(y - ref) <= 1.25 * 2.0 ** -9 * np.linalg.norm(ref)


@pytest.mark.parametrize("M,N,K,sizes", [
    (1, 1, 1, [1]), (1, 128, 128, [1]), (5, 64, 300, [2, 0, 3]), (31, 130, 129, [31]), (40, 256, 512, [3, 7, 0, 30]),
    (200, 100, 256, [150, 50]), (257, 136, 640, [0, 257, 0]), (700, 300, 384, [700]), (900, 513, 200, [400, 500]),
    (1024, 256, 8448, [1024]), (64, 129, 8320, [33, 31])])
def test_grouped_matmul(dev, M, N, K, sizes):
    _close(*_product(np.random.default_rng(M + N + K), dev, M, N, K, sizes))


@pytest.mark.parametrize("M,div", [(48, 8), (300, 2), (900, 8)])
def test_grouped_matmul_gathers_rows(dev, M, div):
    rng = np.random.default_rng(M)
    rows = rng.permutation(M)
    rows[::7] = -1                           # positions that no pair takes
    y, ref, mag = _product(rng, dev, M, 72, 260, [M // 3, 0, M - M // 3], rows, div)
    _close(y, ref, mag)
    assert (y[::7] == 0).all()


@pytest.mark.parametrize("offsets", [[5, 20, 60], [0, 10, 10], [-5, 30, 1000], [50, 20, 70], [0, 0, 0], [80, 90, 100]])
def test_grouped_matmul_offsets_are_brought_into_range(dev, offsets):
    # rows before the first group are nobody's; rows from the last offset on are 0
    rng = np.random.default_rng(1)
    M, N, K = 80, 40, 128
    x = _x(rng, M, K).to(dev)
    w = torch.randn((2, N, K), device=dev) / 11
    xq, xs = ep.ep_quant_rows(x)
    wq, ws = ep.ep_quant_blocks(w)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev)
    ep.ep_grouped_matmul(xq, xs, wq, ws, torch.tensor(offsets, dtype=torch.int32, device=dev), y=y)
    o = [min(max(v, 0), M) for v in offsets]
    xv, _ = R.quant_rows(x.double().cpu().numpy())
    got = y.double().cpu().numpy()
    for g in range(2):
        wv, _ = R.quant_blocks(w[g].double().cpu().numpy())
        i, j = o[g], max(o[g], o[g + 1])
        if g == 0 and offsets == [50, 20, 70]:
            continue                         # empty; the second group owns rows 20 .. 69
        _close(got[i:j], xv[i:j] @ wv.T, np.abs(xv[i:j]) @ np.abs(wv).T)
    assert (got[o[2]:] == 0).all()


def test_grouped_matmul_neighbours_do_not_leak(dev):
    # NaN and infinities of one row, or of another group's weights, stay where they are
    M, N, K = 90, 136, 256
    x = torch.ones((M, K), dtype=torch.bfloat16, device=dev)
    x[40, 7], x[41, 200] = float("nan"), float("inf")
    w = torch.ones((3, N, K), device=dev)
    w[1, 5, 9] = float("nan")
    xq, xs = ep.ep_quant_rows(x)
    wq, ws = ep.ep_quant_blocks(w)
    y = ep.ep_grouped_matmul(xq, xs, wq, ws, torch.tensor([0, 30, 60, 90], dtype=torch.int32, device=dev))
    bad = torch.isnan(y).cpu()
    expect = torch.zeros((M, N), dtype=torch.bool)
    expect[40:42] = True
    expect[30:60, 5] = True
    assert torch.equal(bad, expect)
    assert (y[~bad.to(dev)] == K).all()


def test_grouped_matmul_one_group_without_offsets(dev):
    rng = np.random.default_rng(3)
    x, w = _x(rng, 77, 384).to(dev), torch.randn((1, 50, 384), device=dev) / 20
    xq, xs = ep.ep_quant_rows(x)
    wq, ws = ep.ep_quant_blocks(w)
    a = ep.ep_grouped_matmul(xq, xs, wq, ws)
    b = ep.ep_grouped_matmul(xq, xs, wq, ws, _offsets([77], dev))
    assert torch.equal(a, b)
    assert ep.ep_grouped_matmul(xq[:0], xs[:0], wq, ws).shape == (0, 50)


def test_input_gradient_is_the_product_with_transposed_weights(dev):
    rng = np.random.default_rng(12)
    M, N, K, sizes = 150, 200, 136, [90, 0, 60]
    dy = _x(rng, M, N).to(dev)
    w = torch.from_numpy((rng.normal(0, 0.1, (3, N, K))).astype(np.float32)).to(dev)
    dq, ds = ep.ep_quant_rows(dy)
    wt, wts = ep.ep_quant_blocks(w, transpose=True)
    dx = ep.ep_grouped_matmul(dq, ds, wt, wts, _offsets(sizes, dev)).double().cpu().numpy()
    d, _ = R.quant_rows(dy.double().cpu().numpy())
    for g, (i, j) in enumerate(((0, 90), (90, 90), (90, 150))):
        wv, _ = R.quant_blocks(w[g].double().cpu().numpy())
        _close(dx[i:j], d[i:j] @ wv, np.abs(d[i:j]) @ np.abs(wv))


@pytest.mark.parametrize("M,N,K,sizes", [
    (1, 1, 1, [1]), (5, 8, 8, [5]), (64, 256, 256, [64]), (65, 264, 40, [65]), (130, 100, 33, [130]),
    (200, 72, 300, [10, 0, 190]), (193, 129, 130, [64, 65, 64]), (1000, 520, 264, [400, 600])])
def test_wgrad(dev, M, N, K, sizes):
    rng = np.random.default_rng(M * N)
    dy, x = _x(rng, M, N), _x(rng, M, K)
    out = torch.full((len(sizes), N, K), 7.0, device=dev)
    ep.ep_grouped_wgrad(dy.to(dev), x.to(dev), _offsets(sizes, dev), out=out)
    a, b, i = dy.double().numpy(), x.double().numpy(), 0
    for g, n in enumerate(sizes):
        ref, mag = a[i:i + n].T @ b[i:i + n], np.abs(a[i:i + n]).T @ np.abs(b[i:i + n])
        assert (np.abs(out[g].double().cpu().numpy() - ref) <= (n + 8) * 2.0 ** -24 * mag).all()
        i += n


def test_wgrad_neighbours_do_not_leak_and_strides(dev):
    rng = np.random.default_rng(5)
    dy, x = _x(rng, 100, 200).to(dev), _x(rng, 100, 208).to(dev)
    dy[50:] = float("inf")
    x[50:] = float("nan")
    off = torch.tensor([0, 50, 100], dtype=torch.int32, device=dev)
    for a, b in ((dy[:, :64], x[:, 8:72]), (dy[:, 1:65], x[:, 3:67])):
        g = ep.ep_grouped_wgrad(a, b, off)
        ref = a[:50].double().t() @ b[:50].double()
        mag = a[:50].double().abs().t() @ b[:50].double().abs()
        assert ((g[0].double() - ref).abs() <= 58 * 2.0 ** -24 * mag).all()
        assert torch.isnan(g[1]).all()
    assert (ep.ep_grouped_wgrad(dy[:0], x[:0], torch.zeros(3, dtype=torch.int32, device=dev)) == 0).all()


def test_weight_and_input_gradient_match_differences(dev):
    # L = sum dy * (x w^T) is linear in w and in x: its differences are exact up to rounding
    rng = np.random.default_rng(6)
    M, N, K = 40, 16, 24
    dy = torch.from_numpy(rng.integers(-4, 5, (M, N)).astype(np.float32)).to(torch.bfloat16).to(dev)
    x = torch.from_numpy(rng.integers(-4, 5, (M, K)).astype(np.float32)).to(torch.bfloat16).to(dev)
    w = rng.integers(-4, 5, (1, N, K)).astype(np.float64)
    g = ep.ep_grouped_wgrad(dy, x)[0].cpu().numpy()
    d, a = dy.double().cpu().numpy(), x.double().cpu().numpy()
    loss = lambda w_, a_: (d * (a_ @ w_.T)).sum()
    for n, k in ((0, 0), (3, 20), (15, 23)):
        up = w[0].copy()
        up[n, k] += 1
        assert loss(up, a) - loss(w[0], a) == g[n, k]
    wt, wts = ep.ep_quant_blocks(torch.from_numpy(w.astype(np.float32)).to(dev), transpose=True)
    dq, ds = ep.ep_quant_rows(dy)
    dx = ep.ep_grouped_matmul(dq, ds, wt, wts).double().cpu().numpy()     # small whole numbers: exact
    for m, k in ((0, 0), (17, 5), (39, 23)):
        up = a.copy()
        up[m, k] += 1
        assert loss(w[0], up) - loss(w[0], a) == dx[m, k]


def _layout(dev):
    # 6 experts on 3 ranks, 4 spare slots: slots 0,1 | 4,5 spare of rank 0, ...
    return ep.Layout.create(6, [2, 2, 2], [0, 1, 2, 3, 4, 5], [2, 1, 1], device=dev)


def _slot_rows():
    # physical slot -> (native expert, spare ordinal) of _layout
    return [(0, -1), (1, -1), (-1, 0), (-1, 1), (2, -1), (3, -1), (-1, 2), (4, -1), (5, -1), (-1, 3)]


def test_products_over_physical_slots(dev):
    rng = np.random.default_rng(9)
    lay, M, N, K = _layout(dev), 160, 48, 136
    sizes = [20, 0, 30, 10, 25, 5, 0, 40, 20, 10]
    x, dy = _x(rng, M, K).to(dev), _x(rng, M, N).to(dev)
    w, sw = torch.randn((6, N, K), device=dev) / 10, torch.randn((4, N, K), device=dev) / 10
    (wq, ws), (sq, ss), (xq, xs) = ep.ep_quant_blocks(w), ep.ep_quant_blocks(sw), ep.ep_quant_rows(x)
    off = _offsets(sizes, dev)
    y = ep.ep_grouped_matmul(xq, xs, wq, ws, off, layout=lay, slot_w=sq, slot_w_scale=ss)
    native, slot = ep.ep_grouped_wgrad(dy, x, off, layout=lay)
    one = ep.ep_grouped_wgrad(dy, x, off)
    for s, (e, o) in enumerate(_slot_rows()):
        i, j = int(off[s]), int(off[s + 1])
        a, b = (wq[e:e + 1], ws[e:e + 1]) if e >= 0 else (sq[o:o + 1], ss[o:o + 1])
        if j > i:
            assert torch.equal(y[i:j], ep.ep_grouped_matmul(xq[i:j], xs[i:j].contiguous(), a, b))
        assert torch.equal(native[e] if e >= 0 else slot[o], one[s])


@pytest.mark.parametrize("M,I", [(1, 1), (3, 128), (9, 130), (40, 1536), (5, 77)])
def test_swiglu_quant(dev, M, I):
    # the product rounds once more than its plain form before it is rounded to 8 bits: a value lies within
    # one 8-bit step of the plain one, and all but those next to a boundary are equal
    rng = np.random.default_rng(I)
    x = torch.from_numpy(rng.normal(0, 2, (M, 2 * I)).astype(np.float32)).to(torch.bfloat16)
    q, s = ep.ep_swiglu_quant(x.to(dev))
    a = x.double().numpy()
    h = R.silu(a[:, :I]) * a[:, I:]
    val, e = R.quant_rows(h)
    kb = -(-I // 128)
    got = R.FP8[_bytes(q)] * np.exp2(s.cpu().numpy()[:, :kb].astype(float) - 127).repeat(128, axis=1)
    assert np.array_equal(s.cpu().numpy()[:, :kb], e + 127)
    assert (np.abs(got[:, :I] - h) <= np.abs(h) * 2.0 ** -4 * (1 + 1e-5) + np.exp2(e - 10.0).repeat(128, axis=1)[:, :I] * (1 + 1e-5)).all()
    assert (got[:, :I] != val).mean() < 1e-3
    assert (got[:, I:] == 0).all()


@pytest.mark.parametrize("T,k,H,rows", [(1, 1, 1, 1), (5, 2, 8, 12), (17, 8, 100, 200), (33, 4, 264, 140)])
def test_combine(dev, T, k, H, rows):
    rng = np.random.default_rng(H)
    y = _x(rng, rows, H)
    pos = rng.integers(-2, rows + 2, (T, k)).astype(np.int32)
    pos[0] = -1
    w = rng.normal(0, 1, (T, k)).astype(np.float32)
    out = ep.ep_moe_combine(y.to(dev), torch.from_numpy(pos).to(dev), torch.from_numpy(w).to(dev))
    a, ref, mag = y.double().numpy(), np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < rows:
                ref[t] += w[t, j].astype(np.float64) * a[pos[t, j]]
                mag[t] += abs(w[t, j]) * np.abs(a[pos[t, j]])
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 1) * 2.0 ** -24 * mag).all()
    assert (got[0] == 0).all()


def test_products_repeat_bit_for_bit_and_on_a_side_stream(dev):
    rng = np.random.default_rng(10)
    M, N, K, sizes = 700, 264, 520, [300, 0, 400]
    x, dy = _x(rng, M, K).to(dev), _x(rng, M, N).to(dev)
    w = torch.randn((3, N, K), device=dev)
    off = _offsets(sizes, dev)

    def all_of(stream=None):
        xq, xs = ep.ep_quant_rows(x, stream=stream)
        wq, ws = ep.ep_quant_blocks(w, stream=stream)
        return ep.ep_grouped_matmul(xq, xs, wq, ws, off, stream=stream), ep.ep_grouped_wgrad(dy, x, off, stream=stream)

    a = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = all_of()
    c = all_of(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(a, b, c))
