"""Host-side checks of the gated block, its gradient and the weight gradient of 8-bit rows: bad arguments are refused
before any HIP call (the pointers here are made up)."""
import ctypes
import os

import pytest
import torch

import moe_expert_load_layer_amd as ep
from moe_expert_load_layer_amd import layer as M

pytestmark = pytest.mark.skipif(not os.path.exists(ep.LIB_PATH), reason="library not built")

P = 4096                       # a pointer that no test dereferences
BAD = ep.EP_ERR_INVALID_ARG
BF16, F32, FP8 = ep.EP_DTYPE_BF16, ep.EP_DTYPE_F32, ep.EP_DTYPE_FP8


def _layout():
    return ep._CLayout(12, 8, 16, 4, 5, 2, 1, 0, ctypes.c_void_p(P))


def test_forward_refuses():
    L = ep.lib()
    w = lambda *a: M._CMatrix(*a)  # noqa: E731
    good = w(P, P, 64 * 256, 2)

    def call(**k):
        v = dict(x=P, x_scale=P, x_rows=10, rows=None, rows_div=1, groups=2, offsets=P, m=10, inter=64, k=256, gate=good,
                 up=good, slot_gate=w(), slot_up=w(), layout=None, weights=P, weights_count=10, h=P, h_scale=P,
                 keep_dtype=FP8, keep=P, keep_scale=P)
        v.update(k)
        return L.ep_grouped_swiglu(ctypes.byref(M._CSwiglu(*v.values())), None)

    assert L.ep_grouped_swiglu(None, None) == BAD and call(m=0) == ep.EP_OK
    lay = _layout()
    for bad in (dict(m=-1), dict(m=1 << 31), dict(inter=0), dict(k=0), dict(inter=1 << 25), dict(k=1 << 25),
                dict(groups=0), dict(offsets=None), dict(x=None), dict(x_scale=None), dict(x=P + 8),
                dict(x_scale=P + 2), dict(offsets=P + 2), dict(rows=P + 2), dict(x_rows=9), dict(rows=P, rows_div=0),
                dict(rows=P, x_rows=0), dict(x_rows=1 << 31), dict(h=None), dict(h=P + 8), dict(h_scale=None),
                dict(h_scale=P + 2), dict(weights=P + 2), dict(weights_count=9), dict(weights_count=-1, rows=P),
                dict(keep_dtype=F32), dict(keep=P + 8), dict(keep_scale=None), dict(keep_scale=P + 1),
                dict(keep_dtype=BF16, keep=P + 1), dict(gate=w(None, P, 64 * 256, 2)), dict(up=w(P, None, 64 * 256, 2)),
                dict(up=w(P, P, 64 * 256 - 16, 2)), dict(gate=w(P, P, 64 * 256 + 8, 2)), dict(up=w(P, P, 64 * 256, 1)),
                dict(gate=w(P + 8, P, 64 * 256, 2)), dict(layout=ctypes.pointer(lay)),
                dict(layout=ctypes.pointer(lay), groups=16),
                dict(layout=ctypes.pointer(lay), groups=16, slot_gate=good),
                dict(layout=ctypes.pointer(lay), groups=16, slot_gate=good, slot_up=w(P, P, 64 * 256 - 16, 2))):
        assert call(**bad) == BAD, bad


def test_backward_refuses():
    L = ep.lib()
    need = L.ep_swiglu_backward_workspace_bytes(10, 200)
    assert need == 10 * 2 * 4
    for bad in ((0, 200), (-1, 200), (10, 0), (10, 1 << 25), (1 << 31, 200)):
        assert L.ep_swiglu_backward_workspace_bytes(*bad) == 0
    good = M._CMatrix(P, P, 200 * 256, 4)

    def call(**k):
        v = dict(dy=P, dy_scale=P, dy_rows=10, rows=None, rows_div=1, groups=2, offsets=P, m=10, inter=200, k=256,
                 down=good, slot_down=M._CMatrix(), layout=None, weights=P, weights_count=10, keep_dtype=FP8, keep=P,
                 keep_scale=P, grad=P, q=P, q_scale=P, grad_weights=P, grad_weights_dtype=F32, pos=None, pairs=10, ws=P,
                 ws_bytes=need)
        v.update(k)
        return L.ep_grouped_swiglu_backward(ctypes.byref(M._CSwigluBackward(*v.values())), None)

    assert L.ep_grouped_swiglu_backward(None, None) == BAD
    assert call(m=0, pairs=0) == ep.EP_OK
    for bad in (dict(m=-1), dict(inter=0), dict(k=0), dict(groups=0), dict(offsets=None), dict(dy=None), dict(dy=P + 8),
                dict(dy_scale=None), dict(dy_rows=9), dict(rows=P, rows_div=0), dict(weights=P + 1),
                dict(weights_count=9), dict(keep=None), dict(keep_dtype=F32), dict(keep_scale=None), dict(keep=P + 4),
                dict(keep_dtype=BF16, keep=P + 1), dict(grad=P + 1), dict(q=None), dict(q_scale=None), dict(q=P + 8),
                dict(q_scale=P + 2), dict(grad_weights=P + 2), dict(grad_weights_dtype=FP8), dict(pos=P + 2),
                dict(pairs=9), dict(pairs=-1, pos=P), dict(pairs=1 << 40, pos=P), dict(ws=None), dict(ws=P + 8),
                dict(ws_bytes=need - 1), dict(grad_weights_dtype=BF16, grad_weights=P + 1),
                dict(grad=None, q=None, q_scale=None, grad_weights=None), dict(down=M._CMatrix(P, P, 200 * 256, 3)),
                dict(down=M._CMatrix(P, P, 200 * 256 - 16, 4)), dict(layout=ctypes.pointer(_layout()))):
        assert call(**bad) == BAD, bad


def test_mixed_wgrad_refuses():
    L = ep.lib()
    need = L.ep_wgrad_mixed_workspace_bytes(10, 200)
    assert need == 10 * 256 * 2
    for bad in ((0, 200), (10, 0), (10, 1 << 25), (1 << 31, 200)):
        assert L.ep_wgrad_mixed_workspace_bytes(*bad) == 0

    def call(**k):
        v = dict(dy=P, dy_rows=10, dy_stride=64, x=P, x_scale=P, x_rows=10, dy_places=None, x_places=None, rows_div=1,
                 groups=2, offsets=P, m=10, n=64, k=200, layout=None, out=P, slot_out=None, out_stride=64 * 200,
                 slot_out_stride=0, ws=P, ws_bytes=need)
        v.update(k)
        return L.ep_grouped_wgrad_mixed(ctypes.byref(M._CWgradMixed(*v.values())), None)

    assert L.ep_grouped_wgrad_mixed(None, None) == BAD
    lay = _layout()
    for bad in (dict(m=-1), dict(m=1 << 31), dict(n=0), dict(k=0), dict(groups=0), dict(offsets=None), dict(dy=None),
                dict(dy=P + 1), dict(x=None), dict(x=P + 8), dict(x_scale=None), dict(x_scale=P + 2), dict(out=None),
                dict(out=P + 2), dict(dy_stride=63), dict(dy_stride=1 << 31), dict(dy_rows=9), dict(x_rows=9),
                dict(dy_rows=-1, dy_places=P), dict(x_rows=1 << 31), dict(x_places=P, rows_div=0),
                dict(x_places=P + 2), dict(x_places=P, dy_places=P + 4), dict(x_places=P, dy_places=P, dy_rows=11),
                dict(out_stride=64 * 200 - 1), dict(ws=None), dict(ws=P + 8), dict(ws_bytes=need - 1),
                dict(layout=ctypes.pointer(lay)), dict(layout=ctypes.pointer(lay), groups=16)):
        assert call(**bad) == BAD, bad


def test_python_checks_name_the_argument():
    f, e = torch.zeros, ep.EPBalanceError
    with pytest.raises(e, match="multiple of 128"):
        ep.ep_grouped_swiglu(f(3, 100), f(3, 4), f(1, 8, 100), f(1, 1, 1), f(1, 8, 100), f(1, 1, 1))
    with pytest.raises(e, match="x must be a device tensor"):
        ep.ep_grouped_swiglu(f(3, 128), f(3, 4), f(1, 8, 128), f(1, 1, 1), f(1, 8, 128), f(1, 1, 1))
    with pytest.raises(e, match="multiple of 128"):
        ep.ep_grouped_swiglu_backward(f(3, 128), f(3, 4), f(1, 8, 256), f(1, 1, 2), f(3, 16))
    with pytest.raises(e, match="dy must be a device tensor"):
        ep.ep_grouped_swiglu_backward(f(3, 128), f(3, 4), f(1, 8, 128), f(1, 1, 1), f(3, 16))
    with pytest.raises(e, match="dy must be a device tensor"):
        ep.ep_grouped_wgrad_mixed(f(3, 8), f(3, 128), f(3, 4))
    with pytest.raises(e, match="weights must be \\[pairs\\]"):
        M._pair_weights(f(3, 2), None)
    with pytest.raises(e, match="rows must be \\[output rows\\]"):
        M._places(f(3, 2), "rows")
