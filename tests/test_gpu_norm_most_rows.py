"""The most rows that moe_rmsnorm_e4m3 takes: row numbers stay in 32 bits."""
import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu


def test_rows_up_to_2_31():
    T = 2 ** 31 - 1
    torch.cuda.empty_cache()
    x = torch.empty(T, 1, dtype=torch.bfloat16, device="cuda")
    part = 2 ** 28
    g = torch.Generator(device="cuda").manual_seed(1)
    for a in range(0, T, part):
        x[a:a + part].normal_(generator=g)
    q = torch.empty(T, 1, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(T, 1, device="cuda")
    moe.moe_rmsnorm_e4m3(x, q, scale, normalize=False)
    for a in range(0, T, part):
        v, s = x[a:a + part].float(), scale[a:a + part]
        # two roundings: the constant 1 / 448 and the product with it
        assert bool(((s - v.abs() / 448).abs() <= 2 ** -22 * s).all())
        # a row's only element is its largest: 448 of its scale, or zero
        assert bool((q[a:a + part].float() == 448 * torch.sign(v)).all())
