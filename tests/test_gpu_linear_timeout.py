"""moe_linear whose waits give up: the caller is told, what was started ends, nothing is written, and
the next calls are as before."""
import ctypes as C

import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu

ACT = {"none": 0, "swiglu": 4}
DT = {torch.float32: moe.MOE_DT_F32, torch.bfloat16: moe.MOE_DT_BF16, torch.float16: moe.MOE_DT_F16}


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def given_up(x, w, out, act, offsets, status):
    p = lambda t: None if t is None else C.c_void_p(t.data_ptr())
    R, K = x.shape
    N = out.shape[1]
    E = 0 if offsets is None else offsets.numel() - 1
    s = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    return moe.lib().moe_debug_linear_timeout(
        R, N, K, E, p(x), K, DT[x.dtype], None, p(w), None, None, ACT[act], None, 0, p(offsets),
        p(out), out.stride(0), DT[out.dtype], p(status), s)


# clusters that split K, one CTA a tile (by expert; fp32 sums in registers), pairs of CTAs
@pytest.mark.parametrize("R,N,K,E,od,act", [
    (1, 256, 14336, 0, torch.bfloat16, "none"), (40, 256, 14336, 0, torch.float32, "none"),
    (5, 128, 14336, 0, torch.bfloat16, "swiglu"), (64, 2048, 6144, 16, torch.bfloat16, "swiglu"),
    (64, 2048, 6144, 16, torch.float16, "none"), (2000, 1000, 8192, 0, torch.float32, "none"),
    (5000, 1001, 8192, 0, torch.bfloat16, "none"), (4000, 1008, 8192, 4, torch.bfloat16, "swiglu")])
def test_a_wait_that_gives_up_is_reported(R, N, K, E, od, act):
    rows = 2 * N if act == "swiglu" else N
    dt = torch.float16 if od == torch.float16 else torch.bfloat16
    x, w = randn(1, R, K).to(dt), (randn(2, max(1, E), rows, K) / K ** 0.5).to(dt)
    w = w if E else w[0]
    offsets = torch.linspace(0, R, E + 1, device="cuda").int() if E else None
    wide = torch.full((R + 2, N + 16), 5.0, dtype=od, device="cuda")
    out = wide[1:R + 1, 8:N + 8]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = torch.empty(R, N, dtype=od, device="cuda")
    moe.moe_linear(x, w, want, act=act, offsets=offsets, status=status)
    assert int(status) == moe.MOE_OK
    for _ in range(3):
        status.zero_()
        assert given_up(x, w, out, act, offsets, status) == moe.MOE_OK
        assert int(status) == moe.MOE_ERR_TIMEOUT
        assert bool((wide == 5.0).all())  # nothing is written
    assert given_up(x, w, out, act, offsets, None) == moe.MOE_OK  # without a status
    status.zero_()
    for _ in range(3):  # the tensor memory was given back, and the same bits come out
        out.zero_()
        moe.moe_linear(x, w, out, act=act, offsets=offsets, status=status)
        assert int(status) == moe.MOE_OK and torch.equal(out, want)
