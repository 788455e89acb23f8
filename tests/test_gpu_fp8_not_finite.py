"""Tokens that are not finite through experts with a gate/up clamp: NaN in their rows, nothing in the others."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
import test_gpu_fp8 as t8

pytestmark = pytest.mark.gpu


# streaming kernel (rows quantised by the block; H 8192: by every wave), tiles of 64, 128 and 256 rows
@pytest.mark.parametrize("T,H,I,E,k", [(3, 512, 256, 4, 2), (3, 8192, 128, 4, 2), (40, 512, 256, 4, 2),
                                       (400, 512, 256, 4, 1), (400, 512, 256, 4, 2)])
def test_clamp_keeps_nan(T, H, I, E, k):
    rng, d = np.random.default_rng(T + H), gh.dev()
    w = [torch.from_numpy(v).to(d) for v in t8._layer(rng, H, I, E)]
    ids = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).to(d)
    shape = lib.make_shape(H, I, E, k, T, "bf16", gate_up_limit=0.25)
    off = torch.empty(E + 1, dtype=torch.int32, device=d)
    pairs, pos = (torch.empty(T * k, dtype=torch.int32, device=d) for _ in range(2))
    ws = torch.full((lib.moe_fp8_experts_workspace_bytes(shape),), 0xFF, dtype=torch.uint8, device=d)
    x = gh.to_device_x(t8._x(rng, T, H))
    lib.moe_permute(shape, T, ids, x, off, pairs, pos, x)
    ys = []
    for bad in (0.0, float("nan"), float("inf"), float("-inf")):
        x[1, 200] = bad
        y = torch.empty(T * k, H, dtype=torch.bfloat16, device=d)
        lib.moe_fp8_experts(shape, T, *w, off, pairs, x, y, ws)
        torch.cuda.synchronize()
        ys.append(y.view(T, k, H))
    rest = torch.arange(T, device=d) != 1
    assert bool(torch.isfinite(ys[0]).all())
    for y in ys[1:]:
        assert bool(torch.isnan(y[1]).all()) and torch.equal(y[rest], ys[0][rest])
