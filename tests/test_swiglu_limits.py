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
