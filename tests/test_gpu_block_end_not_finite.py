"""Infinities among a row's last columns, at widths whose columns do not fill a block:
the gradients are those of the formulas, infinities with their signs, NaN where the
formulas have one and nowhere else."""
import numpy as np
import pytest
import torch

import gpu_harness as gh
import mixture_experts_layer_sort_amd as lib
from oracle import block_end

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
INF = float("inf")


def _case(T, H, k, post, nxt):
    g = torch.Generator().manual_seed(T + H + k)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = {"y": n(T * k, H).to(BF), "topk_w": torch.softmax(n(T, k), 1), "shared": n(T, H).to(BF),
         "shared_gate": torch.sigmoid(n(T)), "post_weight": (1 + 0.1 * n(H)).to(BF) if post else None,
         "next_weight": (1 + 0.1 * n(H)).to(BF) if nxt else None, "out": n(T, H).to(BF), "d_out": n(T, H).to(BF),
         "d_normed": n(T, H).to(BF) if nxt else None}
    return a


NAMES = {"d_residual": "d_res", "d_y": "d_y", "d_topk_w": "d_w", "d_shared": "d_shared", "d_gate": "d_gate",
         "d_post_weight": "d_post", "d_next_weight": "d_next"}


def _check(a, T, H, k):
    d = gh.dev()
    t = {n: None if v is None else v.to(d) for n, v in a.items()}
    b = {"d_residual": torch.zeros(T, H, dtype=BF, device=d), "d_y": torch.zeros(T * k, H, dtype=BF, device=d),
         "d_topk_w": torch.zeros(T, k, device=d), "d_shared": torch.zeros(T, H, dtype=BF, device=d),
         "d_gate": torch.zeros(T, device=d)}
    b.update({"d_" + n: torch.zeros(H, device=d) for n in ("post_weight", "next_weight") if a[n] is not None})
    ws = torch.empty(lib.moe_combine_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=d)
    lib.moe_combine_norm_backward(T, H, k, ws=ws, scale=0.5, eps=1e-5, **t, **b)
    torch.cuda.synchronize()
    p = {n: None if v is None else v.double().numpy() for n, v in a.items()}
    with np.errstate(invalid="ignore"):
        ref = block_end.backward(p["y"], p["topk_w"], p["shared"], p["shared_gate"], p["out"], p["post_weight"],
                                 p["next_weight"], 1e-5, 0.5, p["d_out"], p["d_normed"])
    some = 0
    for n, v in b.items():
        g, r = v.double().cpu().numpy(), ref[NAMES[n]][0]
        assert np.array_equal(np.isnan(g), np.isnan(r)), n
        assert np.array_equal(np.isinf(g), np.isinf(r)) and np.array_equal(g[np.isinf(r)], r[np.isinf(r)]), n
        some += np.isinf(r).sum()
    assert some > 0


# 360 and 24 columns of threads short of a block, one, and threads of four chunks; k of either form
SIZES = [(2880, 6), (504, 2), (8, 1), (8200, 3), (2056, 12), (1000, 9)]


@pytest.mark.parametrize("H,k", SIZES)
@pytest.mark.parametrize("nxt", [False, True])
def test_a_row_that_ends_in_an_infinity(H, k, nxt):
    T = 5
    a = _case(T, H, k, False, nxt)
    a["y"][2 * k + k - 1, H - 3], a["y"][3 * k, H - 1] = INF, -INF
    a["shared"][1, H - 8] = -INF
    _check(a, T, H, k)


@pytest.mark.parametrize("H,k", SIZES)
def test_a_gradient_of_the_next_norm_that_ends_in_an_infinity(H, k):
    T = 5
    a = _case(T, H, k, False, True)
    a["d_normed"][2, H - 2], a["d_normed"][4, H - 7] = INF, -INF
    _check(a, T, H, k)


@pytest.mark.parametrize("H,k", SIZES)
def test_a_gradient_that_ends_in_an_infinity_behind_a_norm_of_the_sum(H, k):
    T = 5
    a = _case(T, H, k, True, False)
    a["d_out"][1, H - 1], a["d_out"][3, H - 6] = -INF, INF
    _check(a, T, H, k)
