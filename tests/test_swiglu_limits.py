"""Host-side checks of the gated block at its limits: refused before any HIP call (the pointers here are made up)."""
import ctypes
import os

import pytest

import moe_expert_load_layer_amd as ep
from moe_expert_load_layer_amd import layer as M

pytestmark = pytest.mark.skipif(not os.path.exists(ep.LIB_PATH), reason="library not built")

P = 4096                       # a pointer that no test dereferences
BAD = ep.EP_ERR_INVALID_ARG


def _forward(**k):
    good = M._CMatrix(P, P, 64 * 256, 2)
    v = dict(x=P, x_scale=P, x_rows=10, rows=None, rows_div=1, groups=2, offsets=P, m=10, inter=64, k=256, gate=good,
             up=good, slot_gate=M._CMatrix(), slot_up=M._CMatrix(), layout=None, weights=P, weights_count=10, h=P,
             h_scale=P, keep_dtype=ep.EP_DTYPE_FP8, keep=P, keep_scale=P, sums8=0)
    v.update(k)
    return ep.lib().ep_grouped_swiglu(ctypes.byref(M._CSwiglu(*v.values())), None)


def test_forward_sums():
    assert _forward(m=0) == ep.EP_OK and _forward(m=0, sums8=1) == ep.EP_OK
    for bad in (2, -1, 256):
        assert _forward(sums8=bad) == BAD and _forward(m=0, sums8=bad) == BAD


def _backward(**k):
    v = dict(dy=P, dy_scale=P, dy_rows=10, rows=None, rows_div=1, groups=2, offsets=P, m=10, inter=200, k=256,
             down=M._CMatrix(P, P, 200 * 256, 4), slot_down=M._CMatrix(), layout=None, weights=P, weights_count=10,
             keep_dtype=ep.EP_DTYPE_FP8, keep=P, keep_scale=P, grad=P, q=P, q_scale=P, grad_weights=P,
             grad_weights_dtype=ep.EP_DTYPE_F32, pos=None, pairs=10, ws=P,
             ws_bytes=ep.ep_swiglu_backward_workspace_bytes(10, 200), sums8=0)
    v.update(k)
    return ep.lib().ep_grouped_swiglu_backward(ctypes.byref(M._CSwigluBackward(*v.values())), None)


def test_backward_sums():
    assert _backward(m=0, pairs=0) == ep.EP_OK and _backward(m=0, pairs=0, sums8=1) == ep.EP_OK
    for bad in (2, -1, 256):
        assert _backward(sums8=bad) == BAD and _backward(m=0, pairs=0, sums8=bad) == BAD
