"""Groups of moe_route_logits whose sums are small differences of large scores, against 64 bits."""
import numpy as np
import pytest
import torch
from test_gpu_expert_operators import check_route

pytestmark = pytest.mark.gpu


# E in 8 groups of 2^n lanes and of 20 experts; the biases' size
@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [16, 32, 64, 256, 160])
@pytest.mark.parametrize("size", [1.0, 100.0, 1e4])
def test_groups_whose_biases_cancel(E, size, router):
    """The two best of a group have biases of both signs, and their scores' sums are the same up to
    what fp32 loses of such scores, size 2^-24 each."""
    T, G, k = 600, 8, 4
    gs = E // G
    rng = np.random.default_rng(E + int(size))
    top = 0.9 if router == "sigmoid" else 1.0 / G  # (1 - s(l) is s(-l): sums of 1 would be ties)
    a = rng.uniform(0.2, 0.8, (T, G)) * top
    b = top - a + 2e-8 * size * rng.standard_normal((T, G))
    b = np.clip(b, 0.05 * top, 0.95 * top)
    score = np.full((T, G, gs), 1e-6 * top)
    score[:, :, 0], score[:, :, gs // 2] = a, b
    lg = np.log(score) if router == "softmax" else np.log(score / (1 - score))
    bias = np.full((G, gs), -3.0 * size)
    bias[:, 0], bias[:, gs // 2] = size, -size
    lg = torch.from_numpy(lg.reshape(T, E)).float().cuda()
    bias = torch.from_numpy(bias.reshape(E)).float().cuda()
    for keep in (1, 3, 7):
        check_route(lg, k, bias=bias, router=router, G=G, keep=keep, best=2)


@pytest.mark.parametrize("E", [64, 160])
def test_a_group_of_large_scores_among_small_ones(E):
    """One group's sum is off by far more than the sums at the border, which lie apart."""
    T, G, k, size = 600, 8, 2, 1e4
    gs = E // G
    rng = np.random.default_rng(E)
    sums = 0.5 + 2e-5 * rng.permuted(np.tile(np.arange(G), (T, 1)), axis=1)
    a = rng.uniform(0.2, 0.3, (T, G))
    score = np.full((T, G, gs), 1e-6)
    score[:, :, 0], score[:, :, gs // 2] = a, sums - a
    bias = np.full((G, gs), -3.0)
    bias[:, 0], bias[:, gs // 2] = 1.0, -1.0
    bias[3] *= size
    lg = torch.from_numpy(np.log(score / (1 - score)).reshape(T, E)).float().cuda()
    bias = torch.from_numpy(bias.reshape(E)).float().cuda()
    for keep in (1, 3, 4, 7):
        check_route(lg, k, bias=bias, router="sigmoid", G=G, keep=keep, best=2)
