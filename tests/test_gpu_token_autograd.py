"""The token operators beside autograd: what a call writes counts as written, and gradients through
a torch.autograd.Function are the formula's."""
import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def operands(T=6, k=2, E=4, H=64):
    i32 = dict(dtype=torch.int32, device="cuda")
    ids = (torch.arange(T * k, device="cuda") % E).int().view(T, k)
    off, perm, pos = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T, k, **i32)
    moe.moe_sort_tokens(ids, E, off, perm, pos)
    return ids, off, perm, pos


def test_version_counters_move_on_with_every_output():
    T, k, E, H = 6, 2, 4, 64
    ids, off, perm, pos = operands(T, k, E, H)
    x, y, w = randn(1, T, H), randn(2, T * k, H), randn(3, T, k)
    q, s = torch.empty(T, H, dtype=F8, device="cuda"), torch.empty(T, 1, device="cuda")
    out, res, xs, scs = x.clone(), x.clone(), y.clone(), torch.empty(T * k, 1, device="cuda")
    dy, dw, dx = y.clone(), w.clone(), x.clone()
    wt, prod = randn(4, 32, H).bfloat16(), torch.empty(T, 32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = x.bfloat16()
    for call, written, read in [
            (lambda: moe.moe_rmsnorm_e4m3(x, q, s, resid=res), [q, s, res], [x]),
            (lambda: moe.moe_rmsnorm_e4m3(x, q, s, resid=x), [q, s, x], []),
            (lambda: moe.moe_sort_tokens(ids, E, off, perm, pos), [off, perm, pos], [ids]),
            (lambda: moe.moe_dispatch_rows(x, pos, off, xs, scale=s, scale_s=scs), [xs, scs],
             [x, pos, off, s]),
            (lambda: moe.moe_combine_rows(y, pos, out, w=w), [out], [y, pos, w]),
            (lambda: moe.moe_combine_rows_grad(x, y, pos, off, w, dy, dw), [dy, dw],
             [x, y, pos, off, w]),
            (lambda: moe.moe_dispatch_rows_grad(y, pos, dx), [dx], [y, pos]),
            (lambda: moe.moe_linear(b, wt, prod, status=status), [prod, status], [b, wt])]:
        was = [t._version for t in written + read]
        call()
        now = [t._version for t in written + read]
        assert all(a > b_ for a, b_ in zip(now, was[:len(written)]))
        assert now[len(written):] == was[len(written):]
    with torch.inference_mode():  # such tensors have no counter
        o = torch.empty(T, H, device="cuda")
        moe.moe_combine_rows(y, pos, o, w=w)
    assert torch.equal(o, out)


def test_a_saved_tensor_that_a_call_overwrites_is_noticed():
    _, _, _, pos = operands()
    y = randn(1, 12, 64)
    a = randn(2, 6, 64).requires_grad_()
    other = randn(3, 6, 64)
    z = (a * other).sum()  # backward needs `other`
    moe.moe_combine_rows(y, pos, other)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()


class Combine(torch.autograd.Function):
    """The layer's way back, as a user writes it."""

    @staticmethod
    def forward(ctx, y, w, pos, off):
        out = torch.empty(pos.shape[0], y.shape[1], dtype=y.dtype, device=y.device)
        moe.moe_combine_rows(y, pos, out, w=w)
        ctx.save_for_backward(y, w, pos, off)
        return out

    @staticmethod
    def backward(ctx, dout):
        y, w, pos, off = ctx.saved_tensors
        dy, dw = torch.empty_like(y), torch.empty_like(w)
        moe.moe_combine_rows_grad(dout.contiguous(), y, pos, off, w, dy, dw)
        return dy, dw, None, None


def test_a_function_around_the_calls_trains():
    _, off, _, pos = operands()
    y, w = randn(1, 12, 64).requires_grad_(), randn(2, 6, 2).requires_grad_()
    g = randn(3, 6, 64)
    Combine.apply(y, w, pos, off).backward(g)
    yd, wd = y.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    (yd[pos.long()] * wd[..., None]).sum(1).backward(g.double())
    # one product rounded once; a sum of 64 products in fp32: 2 in a thread's 8, joined by 10 steps
    u = 2.0 ** -24
    assert bool(((y.grad - yd.grad).abs() <= u * yd.grad.abs()).all())
    mag = (yd.detach()[pos.long()] * g.double()[:, None]).abs().sum(-1)
    assert bool(((w.grad - wd.grad).abs() <= 32 * u * mag).all())
