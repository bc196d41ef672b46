"""The layer of e4m3 experts: what it owns and hands to the library's calls (no GPU: the calls are
recorded), and its status word on the GPU."""
import pytest
import torch

import routed_expert_ffn_route_gb300 as moe
from routed_expert_ffn_route_gb300 import e4m3

E, H, I, K = 4, 64, 32, 2
OPERATORS = ("moe_rmsnorm_e4m3", "moe_sort_tokens", "moe_dispatch_rows", "moe_linear",
             "moe_combine_rows")


def layer_on(device, **kw):
    f8 = dict(dtype=torch.float8_e4m3fn, device=device)
    s = dict(dtype=torch.float32, device=device)
    return e4m3.E4m3Experts(torch.zeros(E, 2 * I, H, **f8), torch.ones(E, 2 * I, **s),
                            torch.zeros(E, H, I, **f8), torch.ones(E, H, **s), K, t_max=8, **kw)


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in OPERATORS:
        monkeypatch.setattr(e4m3, name, lambda *a, _n=name, **kw: seen.append((_n, a, kw)))
    return seen


def step(layer, T=5, device="cpu"):
    resid = torch.ones(T, H, dtype=torch.bfloat16, device=device)
    ids = torch.tensor([[0, 3]] * T, dtype=torch.int32, device=device)
    w = torch.full((T, K), 0.5, dtype=torch.float32, device=device)
    return layer.forward(resid, None, ids, w)


def test_both_products_report_to_the_layers_status_word(calls):
    layer = layer_on("cpu")
    step(layer)
    products = [kw for name, _, kw in calls if name == "moe_linear"]
    assert len(products) == 2 and all(kw["status"] is layer.status for kw in products)


def test_reading_the_status_clears_it(calls):
    layer = layer_on("cpu")
    assert layer.read_status() == moe.MOE_OK
    layer.status.fill_(moe.MOE_ERR_TIMEOUT)
    step(layer)  # a later step does not hide it
    assert layer.read_status() == moe.MOE_ERR_TIMEOUT
    assert layer.read_status() == moe.MOE_OK


@pytest.mark.gpu
def test_status_of_a_step_and_of_a_graph():
    layer = layer_on("cuda")
    step(layer, device="cuda")
    assert layer.read_status() == moe.MOE_OK
    resid = torch.ones(5, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[0, 3]] * 5, dtype=torch.int32, device="cuda")
    w = torch.full((5, K), 0.5, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(resid, None, ids, w)
    g.replay()
    assert layer.read_status() == moe.MOE_OK
    layer.status.fill_(moe.MOE_ERR_TIMEOUT)
    g.replay()
    assert layer.read_status() == moe.MOE_ERR_TIMEOUT and layer.read_status() == moe.MOE_OK


@pytest.mark.parametrize("default", [torch.float32, torch.bfloat16, torch.float64])
def test_buffers_do_not_follow_torchs_default_type(default, calls):
    """Scales are fp32 whatever the program's default type is (models often set bf16)."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        layer = layer_on("cpu")
    finally:
        torch.set_default_dtype(before)
    assert {layer.qs.dtype, layer.xss.dtype, layer.hs.dtype} == {torch.float32}
