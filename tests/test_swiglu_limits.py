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


def test_pairs_past_what_a_launch_counts():
    """2^32 - 256 pairs and no more, refused before the gradients are written."""
    most = (1 << 32) - 256
    for pairs in (most + 1, 1 << 38, 1 << 62):
        assert _backward(pairs=pairs, pos=P) == BAD and _backward(m=0, pairs=pairs, pos=P) == BAD


def _mixed(**k):
    v = dict(dy=P, dy_rows=10, dy_stride=64, x=P, x_scale=P, x_rows=10, dy_places=None, x_places=None, rows_div=1,
             groups=2, offsets=P, m=10, n=64, k=200, layout=None, out=P, slot_out=None, out_stride=64 * 200,
             slot_out_stride=0, ws=P, ws_bytes=ep.ep_wgrad_mixed_workspace_bytes(10, 200))
    v.update(k)
    return ep.lib().ep_grouped_wgrad_mixed(ctypes.byref(M._CWgradMixed(*v.values())), None)


def test_rows_past_what_a_launch_counts():
    """Rows in 8 bits: up to (2^24 - 1) * 32 blocks of 128 values."""
    rows, k = 1 << 23, 128 * 65
    assert rows * 65 > (2 ** 24 - 1) * 32
    assert _mixed(x_rows=rows, k=k, out_stride=64 * k, ws_bytes=1 << 62) == BAD
