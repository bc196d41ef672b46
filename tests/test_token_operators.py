"""Refusals of the token operators: every call here returns before any CUDA work, so no GPU
is needed.  Pointers are made-up addresses that are never dereferenced."""
import ctypes as C

import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
F32, BF16, F16, E4M3 = moe.MOE_DT_F32, moe.MOE_DT_BF16, moe.MOE_DT_F16, moe.MOE_DT_E4M3
A = 1 << 20  # an aligned made-up address


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


def call(fn, names, base, **kw):
    bad = set(kw) - set(names)
    assert not bad, bad
    v = dict(base, **kw)
    return fn(*[v[n] for n in names])


NORM = "T H x ldx dt add ldadd w eps norm group resid ldr q ldq scale st".split()
NORM_OK = dict(T=2, H=64, x=A, ldx=64, dt=BF16, add=A, ldadd=64, w=A, eps=1e-6, norm=1, group=32,
               resid=A, ldr=64, q=A, ldq=64, scale=A, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=-4), INVALID), (dict(dt=E4M3), INVALID),
    (dict(dt=9), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID),
    (dict(scale=None), INVALID), (dict(ldx=63), INVALID), (dict(ldq=63), INVALID),
    (dict(ldadd=63), INVALID), (dict(ldr=63), INVALID), (dict(x=A + 1), INVALID),
    (dict(add=A + 1), INVALID), (dict(resid=A + 1), INVALID), (dict(w=A + 1), INVALID),
    (dict(scale=A + 2), INVALID), (dict(dt=F32, x=A + 2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(norm=2), INVALID),
    (dict(H=32769, ldx=40000, ldadd=40000, ldr=40000, ldq=40000), UNSUPPORTED),
    (dict(group=16), UNSUPPORTED), (dict(group=-32), UNSUPPORTED), (dict(group=512), UNSUPPORTED),
    (dict(T=0), moe.MOE_OK)])
def test_norm_refusals(kw, want, L):
    assert call(L.moe_rmsnorm_e4m3, NORM, NORM_OK, **kw) == want


SORT = "T k E ids offsets perm pos st".split()
SORT_OK = dict(T=4, k=2, E=8, ids=A, offsets=A, perm=A, pos=A, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(k=0), UNSUPPORTED), (dict(k=17), UNSUPPORTED),
    (dict(E=0), UNSUPPORTED), (dict(E=257), UNSUPPORTED), (dict(T=65536), UNSUPPORTED),
    (dict(ids=None), INVALID), (dict(offsets=None), INVALID), (dict(perm=None), INVALID),
    (dict(pos=None), INVALID), (dict(ids=A + 2), INVALID), (dict(pos=A + 1), INVALID)])
def test_sort_refusals(kw, want, L):
    assert call(L.moe_sort_tokens, SORT, SORT_OK, **kw) == want


DISP = "T k E H dt x ldx pos offsets xs S sc ldsc scs st".split()
DISP_OK = dict(T=4, k=2, E=8, H=64, dt=BF16, x=A, ldx=64, pos=A, offsets=A, xs=A, S=1, sc=A,
               ldsc=1, scs=A, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(k=17), UNSUPPORTED), (dict(H=0), INVALID), (dict(dt=4), INVALID),
    (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(pos=None), INVALID),
    (dict(offsets=None), INVALID), (dict(ldx=63), INVALID), (dict(x=A + 1), INVALID),
    (dict(S=-1), INVALID), (dict(sc=None), INVALID), (dict(scs=None), INVALID),
    (dict(ldsc=0), INVALID), (dict(scs=A + 2), INVALID), (dict(E=-1), INVALID),
    (dict(T=0), moe.MOE_OK)])
def test_dispatch_refusals(kw, want, L):
    assert call(L.moe_dispatch_rows, DISP, DISP_OK, **kw) == want


COMB = "T k H y ydt pos w add ldadd out ldout odt st".split()
COMB_OK = dict(T=4, k=2, H=64, y=A, ydt=BF16, pos=A, w=A, add=A, ldadd=64, out=A, ldout=64,
               odt=BF16, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(k=0), UNSUPPORTED), (dict(H=0), INVALID), (dict(ydt=E4M3), INVALID),
    (dict(odt=E4M3), INVALID), (dict(odt=F16), UNSUPPORTED), (dict(y=None), INVALID),
    (dict(pos=None), INVALID), (dict(out=None), INVALID), (dict(ldout=63), INVALID),
    (dict(ldadd=63), INVALID), (dict(out=A + 1), INVALID), (dict(w=A + 2), INVALID),
    (dict(T=0), moe.MOE_OK)])
def test_combine_refusals(kw, want, L):
    assert call(L.moe_combine_rows, COMB, COMB_OK, **kw) == want


GRAD = "T k E H dt dout lddout y pos offsets w dy dw st".split()
GRAD_OK = dict(T=4, k=2, E=8, H=64, dt=BF16, dout=A, lddout=64, y=A, pos=A, offsets=A, w=A, dy=A,
               dw=A, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(k=17), UNSUPPORTED), (dict(H=0), INVALID), (dict(dt=E4M3), INVALID),
    (dict(dout=None), INVALID), (dict(y=None), INVALID), (dict(dy=None), INVALID),
    (dict(dw=None), INVALID), (dict(pos=None), INVALID), (dict(offsets=None), INVALID),
    (dict(lddout=63), INVALID), (dict(dw=A + 2), INVALID), (dict(dy=A + 1), INVALID),
    (dict(T=0), moe.MOE_OK)])
def test_combine_grad_refusals(kw, want, L):
    assert call(L.moe_combine_rows_grad, GRAD, GRAD_OK, **kw) == want


DGRAD = "T k H dt dxs pos dx lddx xdt st".split()
DGRAD_OK = dict(T=4, k=2, H=64, dt=BF16, dxs=A, pos=A, dx=A, lddx=64, xdt=BF16, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(dt=E4M3), INVALID), (dict(xdt=F16), UNSUPPORTED),
    (dict(dxs=None), INVALID), (dict(dx=None), INVALID), (dict(lddx=1), INVALID)])
def test_dispatch_grad_refusals(kw, want, L):
    assert call(L.moe_dispatch_rows_grad, DGRAD, DGRAD_OK, **kw) == want


LIN = ("R N K E x ldx dt xs w ws bias act res ldres offsets out ldout odt status st").split()
LIN_OK = dict(R=4, N=32, K=64, E=0, x=A, ldx=64, dt=BF16, xs=None, w=A, ws=None, bias=A, act=0,
              res=A, ldres=32, offsets=None, out=A, ldout=32, odt=BF16, status=None, st=None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(E=-1), INVALID),
    (dict(dt=F32), INVALID), (dict(dt=7), INVALID), (dict(odt=E4M3), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(K=72, ldx=72), UNSUPPORTED),
    (dict(act=4, N=24), UNSUPPORTED), (dict(E=257, offsets=A), UNSUPPORTED),
    (dict(R=(1 << 24) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 1, ldout=1 << 21, ldres=1 << 21),
                                           UNSUPPORTED),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID),
    (dict(ldx=63), INVALID), (dict(ldx=68), INVALID), (dict(ldout=31), INVALID),
    (dict(ldres=31), INVALID), (dict(E=2), INVALID), (dict(x=A + 8), INVALID),
    (dict(w=A + 8), INVALID), (dict(out=A + 1), INVALID), (dict(bias=A + 2), INVALID),
    (dict(status=A + 2), INVALID), (dict(R=0), moe.MOE_OK)])
def test_linear_refusals(kw, want, L):
    assert call(L.moe_linear, LIN, LIN_OK, **kw) == want


def test_binding_checks_its_arguments(L):
    """Shapes, types and strides that the C entry points cannot see raise before the call."""
    f8, i32 = torch.float8_e4m3fn, torch.int32
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, sc = torch.zeros(4, 64, dtype=f8), torch.zeros(4, 1)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_e4m3(x, q[:, :32], sc)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_e4m3(x, q, sc, group=32)           # two groups a row
    with pytest.raises(TypeError):
        moe.moe_rmsnorm_e4m3(x, x, sc)                     # codes must be e4m3
    with pytest.raises(TypeError):
        moe.moe_rmsnorm_e4m3(x.double(), q, sc)
    with pytest.raises(TypeError):
        moe.moe_rmsnorm_e4m3(x, q, sc, add=x.float())
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_e4m3(x.t(), q.t(), torch.zeros(64, 1))
    ids = torch.zeros(4, 2, dtype=i32)
    off, perm = torch.zeros(9, dtype=i32), torch.zeros(8, dtype=i32)
    with pytest.raises(TypeError):
        moe.moe_sort_tokens(ids.long(), 8, off, perm, ids)
    with pytest.raises(ValueError):
        moe.moe_sort_tokens(ids, 4, off, perm, ids)
    xs = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_dispatch_rows(x, ids, off, xs[:7])
    with pytest.raises(ValueError):
        moe.moe_combine_rows(xs[:6], ids, x)
    with pytest.raises(TypeError):
        moe.moe_combine_rows(xs, ids, x, add=x.float())
    with pytest.raises(TypeError):
        moe.moe_combine_rows_grad(x, xs, ids, off, None, xs.float(), torch.zeros(4, 2))
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    out = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_linear(x, w, out, act="swiglu")            # needs 2 N weight rows
    with pytest.raises(ValueError):
        moe.moe_linear(x, w, out, act="tanh")
    with pytest.raises(TypeError):
        moe.moe_linear(x, w.float(), out)
    with pytest.raises(ValueError):
        moe.moe_linear(x, w, out, offsets=off)             # needs w [E, N, K]
    with pytest.raises(ValueError):
        moe.moe_linear(x, w, out, bias=torch.zeros(31))
