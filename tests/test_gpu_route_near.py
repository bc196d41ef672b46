"""The choice of moe_route_logits among scores that fp32 does not tell apart: runs of equal experts
across the last slot, against 64 bits."""
import numpy as np
import pytest
import torch
from test_gpu_expert_operators import check_route

pytestmark = pytest.mark.gpu

# logits this far apart have scores that 64 bits tell apart, and fp32 (softmax) or two floats
# (sigmoid) do not
STEP = {"softmax": 1e-8, "sigmoid": 1e-11}


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
def test_equal_experts_behind_the_last_slot_that_another_pair_moves_up(router):
    """Of 0, 0, d, d the two last are chosen: the second of them is not the first one's shadow."""
    d = STEP[router]
    lg = torch.tensor([[0.0, 0.0, d, d], [0.0, d, d, 0.0], [d, 0.0, 0.0, d]], device="cuda")
    ids, _ = check_route(lg, 2, bias=torch.full((4,), 0.1, device="cuda"), router=router)
    assert ids.tolist() == [[2, 3], [1, 2], [0, 3]]


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
@pytest.mark.parametrize("equal", [2, 3, 4, 5])
def test_equal_experts_across_the_last_slot(router, equal):
    """`equal` experts of one score, some near ones before and behind them, in every order."""
    T, E, d = 400, 64, STEP[router]
    rng = np.random.default_rng(equal)
    lg = np.full((T, E), -4.0)
    for t in range(T):
        levels = [1] * equal + [int(v) for v in rng.choice([0, 1, 2], rng.integers(1, 6))]
        at = rng.choice(E, len(levels), replace=False)
        lg[t, at] = d * rng.permutation(levels)
    lg = torch.from_numpy(lg).float().cuda()
    bias = torch.full((E,), 0.1, device="cuda")
    for k in (1, 2, 3, 4, 6):
        check_route(lg, k, bias=bias, router=router)
        check_route(lg, k, bias=bias, router=router, G=8, keep=3)
        check_route(lg, k, bias=bias, router=router, G=8, keep=3, best=1)
