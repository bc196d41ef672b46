"""The operators between router and experts: streams that a call is given, groups of SwiGLU beside one
with a NaN or an infinity, and fp32 sums of 8-bit integers past one chunk of K."""
import math

import pytest
import torch
from test_gpu_expert_operators import (T32, TB, TH, U, check_glu, check_glu_grad, codes, glu_buffers,
                                       randn)

import routed_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu


def test_calls_run_on_the_stream_that_they_are_given():
    """The current stream is busy for some 50 ms meanwhile: what ran there would come too late."""
    T, E, k, I, N, K = 37, 64, 6, 256, 96, 256
    lg, dw, z, dh = randn(1, T, E), randn(2, T, k), randn(3, T, 2 * I, dtype=TB), randn(4, T, I, dtype=TB)
    x, w = codes(5, T, K), codes(6, N, K)
    pos = torch.randperm(T, device="cuda").int()[:, None].contiguous()
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def outputs():
        h, q, sc = glu_buffers(T, I, 128, TB)
        return dict(ids=torch.full((T, k), 77, dtype=torch.int32, device="cuda"),
                    w=torch.full((T, k), 77.0, device="cuda"), dl=torch.full_like(lg, 77.0), h=h, q=q,
                    sc=sc, dz=torch.full_like(z, 77.0), xs=torch.full_like(x, 77),
                    out=torch.full((T, N), 77.0, device="cuda"))

    def calls(o, stream):
        moe.moe_route_logits(lg, o["ids"], o["w"], router="sigmoid", stream=stream)
        moe.moe_route_logits_grad(dw, lg, o["ids"], o["dl"], router="sigmoid", stream=stream)
        moe.moe_swiglu_e4m3(z, o["h"], o["q"], o["sc"], stream=stream)
        moe.moe_swiglu_e4m3_grad(dh, o["q"], o["sc"], o["dz"], stream=stream)
        moe.moe_dispatch_rows(x, pos, off, o["xs"], stream=stream)
        moe.moe_linear(x, w, o["out"], stream=stream)

    want, got = outputs(), outputs()
    calls(want, None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = {n: t.cpu() for n, t in want.items()}
    busy = torch.cuda.Event()
    torch.cuda._sleep(100_000_000)
    busy.record()
    calls(got, s)
    with torch.cuda.stream(s):
        got = {n: t.cpu() for n, t in got.items()}
    assert not busy.query()  # else the test says nothing
    for n in want:
        assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), n
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [TB, TH, T32])
@pytest.mark.parametrize("I", [256, 252, 250, 255])  # words of eight, four, two and one
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("half", [0, 1])
def test_swiglu_of_a_group_leaves_the_others(I, dtype, bad, half):
    R, group = 5, 128
    z, dh = randn(1, R, 2 * I, dtype=dtype, scale=2), randn(2, R, I, dtype=dtype)
    z[1, half * I + 5] = bad
    z[3, half * I + group - 1] = bad
    h, q, scale = glu_buffers(R, I, group, dtype)
    moe.moe_swiglu_e4m3(z, h, q, scale, group=group)
    dz, h2 = torch.full_like(z, 5), torch.full_like(dh, 5)
    moe.moe_swiglu_e4m3_grad(dh, q, scale, dz, h=h2, group=group)

    def part(t, a, b):  # columns a .. b of both halves
        return torch.cat([t[:, a:b], t[:, I + a:I + b]], 1)

    n = I - group  # the second group of each half
    check_glu(part(z, group, I), n, group, h[:, group:], part(q, group, I), scale[:, [1, 3]])
    check_glu_grad(dh[:, group:], part(q, group, I), scale[:, [1, 3]], group, part(dz, group, I),
                   h2[:, group:])
    ok = [0, 2, 4]
    check_glu(z[ok], I, group, h[ok], q[ok], scale[ok])
    check_glu_grad(dh[ok], q[ok], scale[ok], group, dz[ok], h2[ok])
    # of the group itself h has the exact z, and the other half its own scale
    cols = torch.arange(I, device="cuda") != 5
    cols[group - 1] = False
    assert bool(torch.isfinite(h[:, cols].float()).all())
    assert bool(torch.isfinite(scale[:, [2 * (1 - half), 2 * (1 - half) + 1]]).all())
    assert not bool(torch.isfinite(scale[[1, 3], 2 * half]).any())


# few rows, clusters that split K, one CTA a tile
@pytest.mark.parametrize("R,N,K", [(3, 96, 6144), (8, 512, 14336), (24, 512, 6144), (40, 256, 14336),
                                   (130, 700, 3840), (700, 513, 4096), (2000, 1000, 8192)])
def test_integer_product_fp32_sums_past_one_chunk(R, N, K):
    """fp32 outputs: whole numbers below 2^24 are exact whatever K; larger sums are rounded to nearest
    once every 1024 of K and once for each other CTA of a cluster, of eight at most."""
    g = torch.Generator(device="cuda").manual_seed(R)

    def draw(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int8)

    out = torch.empty(R, N, device="cuda")
    x, w = draw(-30, 31, R, K), draw(-30, 31, N, K)  # 900 K < 2^24
    moe.moe_linear(x, w, out)
    assert torch.equal(out.double(), x.double() @ w.double().t())
    # of one sign: every cut-off sum would be too small by some 2^-25 a step of 16 of K
    x, w = draw(90, 128, R, K), draw(90, 128, N, K)
    moe.moe_linear(x, w, out)
    ref = x.double() @ w.double().t()
    err = (out.double() - ref).abs()
    assert bool((err <= (-(-K // 1024) + 8) * U * ref).all()), float((err / ref).max())
