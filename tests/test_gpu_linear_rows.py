"""moe_linear on rows that lie at odd distances where there is no next row."""
import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float8_e4m3fn])
@pytest.mark.parametrize("gap", [1, 3, 8])
def test_one_row_at_any_distance(dtype, gap):
    """The distance to the next row has no meaning for a single one."""
    N, K = 48, 64
    g = torch.Generator(device="cuda").manual_seed(gap)
    wide = torch.randn(2, K + gap, generator=g, device="cuda").to(dtype)
    w = torch.randn(N, K, generator=g, device="cuda").to(dtype)
    x = wide[:1, :K]
    assert x.stride(0) == K + gap
    out, want = torch.empty(1, N, device="cuda"), torch.empty(1, N, device="cuda")
    moe.moe_linear(x, w, out)
    moe.moe_linear(x.clone(memory_format=torch.contiguous_format), w, want)
    assert torch.equal(out, want)


def test_more_rows_at_odd_distances_are_refused():
    wide = torch.zeros(2, 67, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(48, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoEError) as e:
        moe.moe_linear(wide[:, :64], w, torch.empty(2, 48, device="cuda"))
    assert e.value.status == moe.MOE_ERR_INVALID_ARG
