"""Groups of softmax scores behind logits so large that one less 80 is the same number, +inf (which
counts as the largest finite number) among them: all other scores are 0, whose ties go by index.  And
scores smaller than two floats tell apart."""
import numpy as np
import pytest
import torch
from test_gpu_expert_operators import T32, TB, check_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [T32, TB])
@pytest.mark.parametrize("top", [1e6, 1e9, 3e9, 1e20, float("inf")])
@pytest.mark.parametrize("E,G", [(32, 8), (64, 4), (128, 8), (256, 8), (60, 6)])
def test_softmax_groups_behind_large_logits(E, G, top, dtype):
    T, k = 60, 6
    rng = np.random.default_rng(E)
    lg = rng.standard_normal((T, E))
    lg[rng.random((T, E)) < 0.9] = -np.inf  # groups of none, one, or a few
    for t in range(T):
        lg[t, rng.choice(E, 1 + t % 3, replace=False)] = top
    lg = torch.from_numpy(lg).to(dtype).cuda()
    if top == float("inf"):
        lg[0, 0] = torch.finfo(T32).max if dtype == T32 else torch.finfo(TB).max
    for keep in (1, 2, 3):
        for best in (1, 2):
            check_route(lg, k, router="softmax", G=G, keep=keep, best=best)
            check_route(lg, k, router="sigmoid", G=G, keep=keep, best=best)
            check_route(lg, k, router="softmax", bias=torch.zeros(E, device="cuda"), G=G, keep=keep,
                        best=best)


@pytest.mark.parametrize("E,G", [(32, 8), (64, 4), (256, 8)])
def test_softmax_groups_of_very_small_scores(E, G):
    """Scores of 1e-35 to 1e-48 beside larger ones: what a group's are decides, not how many it has."""
    T, k = 200, 6
    rng = np.random.default_rng(E)
    lg = rng.uniform(-110.0, -82.0, (T, E))
    lg[rng.random((T, E)) < 0.9] = -np.inf
    lg[np.arange(T), rng.choice(E, T)] = 0.0
    lg = torch.from_numpy(lg).float().cuda()
    for keep in (1, 2, 3):
        for best in (1, 2):
            check_route(lg, k, router="softmax", G=G, keep=keep, best=best)
