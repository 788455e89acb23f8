"""Every finite number is one (no GPU is touched: no tokens)."""
import ctypes
import math

import numpy as np
import pytest

import mixture_experts_layer_sort_amd as lib

OK, INVALID = 0, -1
TOP = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("v,status", [(TOP, OK), (-TOP, OK), (3.1e38, OK), (-3.3e38, OK), (0.0, OK), (math.inf, INVALID),
                                      (-math.inf, INVALID), (math.nan, INVALID)])
def test_scales_and_eps(v, status):
    so = lib.load()
    r = lib.make_router(64, 4, "sigmoid", scale=v)
    assert so.moe_route_scores(ctypes.byref(r), 0, None, 64, None, None, None, None) == status
    assert so.moe_route_scores_backward(ctypes.byref(r), 0, None, 64, None, None, None, 0, None, 64, None) == status
    none = [None] * 7
    assert so.moe_combine_norm(0, 64, 1, *none, 1e-6, v, None, None, None) == status
    assert so.moe_combine_norm_backward(0, 64, 1, *none, 1e-6, v, *[None] * 9, None, 0, None) == status
    eps = INVALID if v < 0 else status
    assert so.moe_combine_norm(0, 64, 1, *none, v, 1.0, None, None, None) == eps
    assert so.moe_combine_norm_backward(0, 64, 1, *none, v, 1.0, *[None] * 9, None, 0, None) == eps
