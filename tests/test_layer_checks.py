"""Host-side checks of the operators around the balancer, without a GPU: bad arguments are refused before any HIP
call (the pointers here are made up)."""
import ctypes
import os

import pytest
import torch

import moe_expert_load_layer_amd as ep
from moe_expert_load_layer_amd import layer as M

pytestmark = pytest.mark.skipif(not os.path.exists(ep.LIB_PATH), reason="library not built")

P = 4096                       # a pointer that no test dereferences
BAD = ep.EP_ERR_INVALID_ARG


def gate(**k):
    v = dict(num_experts=16, top_k=4, num_groups=1, topk_groups=1, logits_dtype=0, scale=1.0, bias=None)
    v.update(k)
    return M._CGate(*v.values())


def test_gate_refuses():
    L = ep.lib()
    call = lambda g, logits=P, stride=16, T=3, ids=P, w=P: L.ep_gate_topk(  # noqa: E731
        logits, stride, T, ctypes.byref(g), ids, w, None)
    assert call(gate(), T=0) == ep.EP_OK                      # nothing to do
    for bad in (dict(num_experts=0), dict(num_experts=1025), dict(top_k=0), dict(top_k=17), dict(top_k=17, num_experts=17),
                dict(num_groups=3), dict(num_groups=0), dict(num_groups=4, topk_groups=5), dict(topk_groups=0),
                dict(num_groups=32, num_experts=64), dict(logits_dtype=2), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(bias=P + 2), dict(num_experts=2)):
        assert call(gate(**bad), stride=2048) == BAD, bad
    assert call(gate(), stride=15) == BAD
    assert call(gate(), T=-1) == BAD
    assert call(gate(), logits=None) == BAD and call(gate(), ids=None) == BAD and call(gate(), w=None) == BAD
    assert call(gate(), logits=P + 2) == BAD and call(gate(), ids=P + 1) == BAD
    assert L.ep_gate_topk(P, 16, 3, None, P, P, None) == BAD
    back = lambda g, ids=P, w=P, d=P, T=3, out=P: L.ep_gate_topk_backward(  # noqa: E731
        ids, w, d, T, ctypes.byref(g), out, None)
    assert back(gate(), T=0) == ep.EP_OK
    assert back(gate(top_k=0)) == BAD and back(gate(), ids=None) == BAD and back(gate(), out=P + 2) == BAD
    assert back(gate(), T=-1) == BAD


def test_quantisation_refuses():
    L = ep.lib()
    rows = lambda x=P, dt=1, m=4, k=200, st=200, q=P, s=P: L.ep_quant_rows(x, dt, m, k, st, q, s, None)  # noqa: E731
    assert rows(m=0) == ep.EP_OK
    for bad in (dict(dt=2), dict(m=-1), dict(k=0), dict(st=199), dict(x=None), dict(q=None), dict(s=None),
                dict(x=P + 1), dict(q=P + 8), dict(s=P + 2), dict(m=1 << 41), dict(k=1 << 25, st=1 << 25)):
        assert rows(**bad) == BAD, bad
    blocks = lambda w=P, dt=0, g=2, gs=600, n=20, k=30, q=P, s=P: L.ep_quant_blocks(  # noqa: E731
        w, dt, g, gs, n, k, 0, q, s, None)
    assert blocks(g=0) == ep.EP_OK
    for bad in (dict(dt=2), dict(g=-1), dict(g=70000), dict(gs=599), dict(n=0), dict(k=0), dict(w=None), dict(q=None),
                dict(s=None), dict(w=P + 2), dict(q=P + 4)):
        assert blocks(**bad) == BAD, bad
    glu = lambda x=P, m=4, i=64, q=P, s=P: L.ep_swiglu_quant(x, m, i, q, s, None)  # noqa: E731
    assert glu(m=0) == ep.EP_OK
    for bad in (dict(m=-1), dict(i=0), dict(x=None), dict(q=P + 8), dict(s=P + 1), dict(x=P + 1)):
        assert glu(**bad) == BAD, bad
    comb = lambda y=P, r=9, p=P, w=P, t=3, k=2, h=8, o=P: L.ep_moe_combine(y, r, p, w, t, k, h, o, None)  # noqa: E731
    assert comb(t=0) == ep.EP_OK
    for bad in (dict(y=None), dict(r=-1), dict(p=None), dict(w=None), dict(t=-1), dict(k=0), dict(h=0), dict(o=None),
                dict(p=P + 2), dict(o=P + 1)):
        assert comb(**bad) == BAD, bad


def _layout():
    return ep._CLayout(12, 8, 16, 4, 5, 2, 1, 0, ctypes.c_void_p(P))


def test_products_refuse():
    L = ep.lib()

    def matmul(**k):
        p = M._CMatmul(P, P, 10, None, 1, 2, P, 10, 64, 256, M._CMatrix(P, P, 64 * 256, 2), M._CMatrix(), None, P)
        for f, v in k.items():
            setattr(p, f, v)
        return L.ep_grouped_matmul(ctypes.byref(p), None)

    assert matmul(m=0) == ep.EP_OK
    assert L.ep_grouped_matmul(None, None) == BAD
    lay = _layout()
    for bad in (dict(m=-1), dict(m=1 << 31), dict(n=0), dict(k=0), dict(groups=0), dict(offsets=None), dict(x=None),
                dict(x_scale=None), dict(y=None), dict(x=P + 8), dict(x_scale=P + 2), dict(y=P + 1),
                dict(offsets=P + 2), dict(rows=P + 2), dict(x_rows=9), dict(rows=P, rows_div=0), dict(rows=P, x_rows=0),
                dict(w=M._CMatrix(None, P, 64 * 256, 2)), dict(w=M._CMatrix(P, None, 64 * 256, 2)),
                dict(w=M._CMatrix(P, P, 64 * 256 - 16, 2)), dict(w=M._CMatrix(P, P, 64 * 256 + 8, 2)),
                dict(w=M._CMatrix(P, P, 64 * 256, 1)), dict(w=M._CMatrix(P + 8, P, 64 * 256, 2)),
                dict(layout=ctypes.pointer(lay)),                                     # 2 groups, 16 slots
                dict(layout=ctypes.pointer(lay), groups=16)):                         # no spare slots' weights
        assert matmul(**bad) == BAD, bad

    def wgrad(**k):
        p = M._CWgrad(P, P, 64, 256, 10, 64, 256, 2, P, None, P, None, 64 * 256, 0)
        for f, v in k.items():
            setattr(p, f, v)
        return L.ep_grouped_wgrad(ctypes.byref(p), None)

    assert L.ep_grouped_wgrad(None, None) == BAD
    for bad in (dict(m=-1), dict(m=1 << 31), dict(n=0), dict(k=0), dict(groups=0), dict(offsets=None), dict(dy=None),
                dict(x=None), dict(out=None), dict(dy=P + 1), dict(out=P + 2), dict(dy_stride=63), dict(x_stride=255),
                dict(out_stride=64 * 256 - 1), dict(layout=ctypes.pointer(lay)),
                dict(layout=ctypes.pointer(lay), groups=16)):
        assert wgrad(**bad) == BAD, bad


def test_few_tokens_refuses():
    L = ep.lib()
    E, H, I, T, k = 16, 64, 32, 3, 4
    bytes_ = L.ep_few_tokens_workspace_bytes(T, k, H, I)
    assert bytes_ >= T * k * I * 4
    for bad in ((65, k, H, I), (-1, k, H, I), (T, 17, H, I), (T, 0, H, I), (T, k, H + 4, I), (T, k, H, 0),
                (T, k, 1 << 17, I)):
        assert L.ep_few_tokens_workspace_bytes(*bad) == 0, bad

    def call(x=P, xs=H, T=T, logits=P, ls=E, g=None, e=None, out=P, os_=H, ids=P, w=P, ws=P, n=bytes_):
        g = gate() if g is None else g
        e = experts() if e is None else e
        return L.ep_moe_few_tokens(x, xs, T, logits, ls, ctypes.byref(g), ctypes.byref(e), out, os_, ids, w, ws, n, None)

    def experts(hidden=H, inter=I, dtype=1, **k):
        fp8 = dtype == 2
        m = lambda n, kk: M._CMatrix(P, P if fp8 else None, n * (128 if fp8 else 2 * kk), 1)  # noqa: E731
        v = dict(gate=m(I, H), up=m(I, H), down=m(H, I))
        v.update(k)
        return M._CExperts(hidden, inter, dtype, v["gate"], v["up"], v["down"])

    assert call(T=0) == ep.EP_OK and call(T=0, e=experts(dtype=2)) == ep.EP_OK
    for bad in (dict(T=65), dict(T=-1), dict(x=None), dict(x=P + 2), dict(xs=H - 8), dict(xs=H + 4), dict(logits=None),
                dict(ls=E - 1), dict(out=None), dict(os_=H - 1), dict(ids=None), dict(w=None), dict(ws=None),
                dict(ws=P + 8), dict(n=bytes_ - 1), dict(g=gate(top_k=0)), dict(e=experts(hidden=60)),
                dict(e=experts(inter=4)), dict(e=experts(dtype=0)),
                dict(e=experts(up=M._CMatrix(None, None, I * H * 2, 0))),
                dict(e=experts(down=M._CMatrix(P, None, I * H * 2 - 16, 0))),
                dict(e=experts(gate=M._CMatrix(P, None, I * H * 2 + 2, 0))),
                dict(e=experts(gate=M._CMatrix(P + 2, None, I * H * 2, 0))),
                dict(e=experts(dtype=2, gate=M._CMatrix(P, None, I * 128, 1))),
                dict(e=experts(dtype=2, gate=M._CMatrix(P, P, I * 128, 0)))):
        assert call(**bad) == BAD, bad


def test_adamw_refuses():
    L = ep.lib()

    def step(t=(P, P, P, P, P, P, None, 100), n=1, **k):
        words = (ctypes.c_int64 * 8)(*[0 if v is None else v for v in t])
        v = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, grad_scale=1.0, step=1, seed=0, bits=32,
                 dtype=0)
        v.update(k)
        return L.ep_adamw_step(words, n, ctypes.byref(M._CAdamW(*v.values())), None)

    ok = (P, P, P, P, P, P, None, 0)
    assert step(t=ok) == ep.EP_OK and step(n=0) == ep.EP_OK      # nothing to do
    nan = float("nan")
    for bad in (dict(step=0), dict(bits=16), dict(dtype=2), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
                dict(beta2=nan), dict(eps=-1.0), dict(lr=nan), dict(weight_decay=float("inf")), dict(grad_scale=nan),
                dict(n=-1), dict(t=(None, P, P, P, P, P, None, 100)), dict(t=(P, None, P, P, P, P, None, 100)),
                dict(t=(P, P, None, P, P, P, None, 100)), dict(t=(P, P, P, None, P, P, None, 100)),
                dict(t=(P + 2, P, P, P, P, P, None, 100)), dict(t=(P, P + 2, P, P, P, P, None, 100)),
                dict(t=(P, P, P + 1, P, P, P, None, 100)), dict(t=(P, P, P, P, P, P, P + 1, 100)),
                dict(t=(P, P, P, P, P, P, None, -1)), dict(t=(P, P, P, P, P, P, None, 1 << 50)),
                dict(bits=8, t=(P, P, P, P, None, P, None, 100)), dict(bits=8, t=(P, P, P, P, P, None, None, 100))):
        assert step(**bad) == BAD, bad
    assert L.ep_adamw_step(None, 1, ctypes.byref(M._CAdamW(1e-3, .9, .99, 1e-8, 0, 1, 1, 0, 32, 0)), None) == BAD
    one = (ctypes.c_int64 * 8)(P, 0, P, P, P, P, 0, 100)
    nul, ptr = (ctypes.c_void_p * 1)(None), (ctypes.c_void_p * 1)(P)
    assert L.ep_adamw_values(one, 1, nul, ptr, None) == BAD and L.ep_adamw_values(None, 1, ptr, ptr, None) == BAD


def test_python_checks_name_the_argument():
    # host tensors, wrong types and shapes are refused before the library is called
    f = torch.zeros
    with pytest.raises(ep.EPBalanceError, match="logits must be a device tensor"):
        ep.ep_gate_topk(f(3, 8), 2)
    with pytest.raises(ep.EPBalanceError, match="ids must be"):
        ep.ep_gate_topk_backward(f(4, dtype=torch.int32), f(4), f(4), 8)
    with pytest.raises(ep.EPBalanceError, match="float32 or bfloat16"):
        ep.ep_gate_topk_backward(f(4, 2, dtype=torch.int32), f(4, 2), f(4, 2), 8, dtype=torch.float16)
    with pytest.raises(ep.EPBalanceError, match="x must be a device tensor"):
        ep.ep_quant_rows(f(3, 8))
    with pytest.raises(ep.EPBalanceError, match="w must be a device tensor"):
        ep.ep_quant_blocks(f(3, 8, 8))
    with pytest.raises(ep.EPBalanceError, match="2 \\* inter"):
        ep.ep_swiglu_quant(f(3, 7))
    with pytest.raises(ep.EPBalanceError, match="multiple of 128"):
        ep.ep_grouped_matmul(f(3, 100), f(3, 4), f(1, 8, 100), f(1, 1, 1))
    with pytest.raises(ep.EPBalanceError, match="dy must be a device tensor"):
        ep.ep_grouped_wgrad(f(3, 8), f(3, 8))
    with pytest.raises(ep.EPBalanceError, match="x must be a device tensor"):
        ep.ep_moe_few_tokens(f(3, 8), f(3, 4), 2, f(4, 8, 8), f(4, 8, 8), f(4, 8, 8))
    with pytest.raises(ep.EPBalanceError, match="bits must be"):
        ep.AdamW([], bits=16)
    with pytest.raises(ep.EPBalanceError, match="params\\[0\\] must be a device tensor"):
        ep.AdamW([f(3)])
    assert ep.ep_scale_stride(0) == 0 and ep.ep_scale_stride(1) == 4 and ep.ep_scale_stride(513) == 8
