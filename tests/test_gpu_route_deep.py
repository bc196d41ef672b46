"""Weights and gradients of renormalised sigmoids whose logits lie far below 0, some of them or all,
relative to each weight's own size, against 64 bits."""
import pytest
import torch
from test_gpu_expert_operators import T32, TB, TH, check_grad, check_route, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [T32, TB, TH])
@pytest.mark.parametrize("top", [-59.0, -30.0, -61.0, 0.5, 20.0, -200.0])
def test_sigmoids_of_deep_logits(top, dtype):
    T, E, k = 40, 32, 6
    lg = (top - 60.0 * torch.rand(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    lg[::3, 0] = top
    lg[1::3, 4:] = -float("inf")  # empty slots beside them
    lg = lg.to(dtype)
    for norm in (True, False):
        ids, w = check_route(lg, k, router="sigmoid", norm=norm, f=2.5)
        check_grad(randn(2, T, k), lg, ids, "sigmoid", norm, 2.5)
    check_route(lg, k, router="softmax")
