"""A layer of e4m3 experts behind the library's router, against the same layer in 64 bits."""
import pytest
import torch

import gen
import routed_expert_ffn_route_gb300 as moe
from gen.device import build_packed_layer
from routed_expert_ffn_route_gb300.e4m3 import E4m3Experts, quantize_e4m3

pytestmark = pytest.mark.gpu


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def routed(spec, cfg, packed, x):
    T = x.shape[0]
    ids = torch.empty((T, spec.top_k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, spec.top_k), device="cuda")
    ws = torch.zeros(moe.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    moe.moe_route_topk(cfg, packed, x, ids, w, ws)
    assert moe.moe_read_status(ws) == moe.MOE_OK
    return ids, w


@pytest.mark.parametrize("T", [1, 7, 64, 301])
@pytest.mark.parametrize("top_p", [0.0, 0.6])
def test_layer_matches_64_bits(T, top_p):
    spec = gen.LayerSpec("e4m3", hidden=512, inter=256, n_experts=16, top_k=4,
                         router="sigmoid_grouped", n_group=4, topk_group=2, rsf=2.5, bias_std=0.1)
    cfg, packed = build_packed_layer(spec, 0, 0, "cuda", host_codes=True)
    cfg.expert_top_p = top_p
    E, H, I = spec.n_experts, spec.hidden, spec.inter
    w1, s1 = quantize_e4m3(randn(1, E, 2 * I, H) / H ** 0.5)
    w2, s2 = quantize_e4m3((randn(2, E, H, I) / I ** 0.5).bfloat16())
    norm = (1 + 0.1 * randn(3, H)).bfloat16()
    resid, add = randn(4, T, H).bfloat16(), randn(5, T, H).bfloat16()
    layer = E4m3Experts(w1, s1, w2, s2, spec.top_k, t_max=512, norm_weight=norm)
    ids, w = routed(spec, cfg, packed, resid)
    if top_p:
        assert bool((ids < 0).any()) or T == 1
    out = layer.forward(resid, add, ids, w).clone()

    # 64 bits, with the roundings that the layer's types make: the codes of x are taken from the
    # layer (its own test bounds them), h is rounded to bf16 and to e4m3 where it differs
    r = (resid.float() + add.float()).bfloat16().double()
    x = layer.q[:T].double() * layer.qs[:T].double()
    W1, W2 = w1.double() * s1.double()[..., None], w2.double() * s2.double()[..., None]
    ref, err = r.clone(), torch.zeros_like(r)
    for j in range(spec.top_k):
        for e in range(E):
            t = torch.nonzero(ids[:, j] == e)[:, 0]
            if not len(t):
                continue
            z = x[t] @ W1[e].t()
            h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
            wj = w[t, j, None].double()
            y = h @ W2[e].t()
            ref[t] += wj * y
            # h: half a step of bf16, then of e4m3 (2^-4 of the value, or 2^-10 of its row's
            # scale near zero), in every product; y: half a step of bf16 on top
            step = h.abs() * (2 ** -8 + 2 ** -4) + h.abs().amax(1, keepdim=True) / 448 * 2 ** -10
            dy = step @ W2[e].abs().t()
            err[t] += wj.abs() * (dy + 2 ** -8 * (y.abs() + dy))
    off = (out.double() - ref).abs()
    # what every element may be off at most, the output's rounding, and fp32 in between
    assert bool((off <= (err + 2 ** -8 * (ref.abs() + err)) * (1 + 2 ** -10) + 2 ** -18).all())
    # errors of h are independent of one another: in the norm they stay near e4m3's own
    # root-mean-square error, at most 2^-4 / sqrt(3); h, y and the output round to bf16
    bf16 = 2 ** -8 * (2 + float(ref.norm() / (ref - r).norm()))
    assert float(off.norm() / (ref - r).norm()) < 2 ** -4 / 3 ** 0.5 + bf16
    assert layer.forward(resid, add, ids, w).equal(out)


def test_quantiser_and_room():
    q, s = quantize_e4m3(randn(1, 3, 5, 64))
    assert q.shape == (3, 5, 64) and s.shape == (3, 5)
    w1, s1 = quantize_e4m3(randn(2, 2, 64, 64))
    w2, s2 = quantize_e4m3(randn(3, 2, 64, 32))
    layer = E4m3Experts(w1, s1, w2, s2, 2, t_max=4)
    with pytest.raises(ValueError):
        layer.forward(randn(4, 5, 64).bfloat16(), None, None, None)
    with pytest.raises(ValueError):
        E4m3Experts(w1, s1, w2[:, :, :16].contiguous(), s2, 2, t_max=4)
