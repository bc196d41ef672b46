"""Token operators on the GPU against plain forms in 64 bits.

Tolerances: u = 2^-24 is half a step of fp32; a value rounded to a type t once is off by at
most finfo(t).eps / 2 of itself; e4m3: 2^-4, or 2^-10 below its smallest normal number.
"""
import math

import numpy as np
import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
T32, TB, TH = torch.float32, torch.bfloat16, torch.float16


def randn(seed, *shape, dtype=T32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = d > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, worst {float((d - tol).max()):.3g}"


# ------------------------------------------------------------------------ norm to e4m3
def norm_ref(x, add, w, eps, group, normalize):
    r = (x.float() + add.float()).to(x.dtype) if add is not None else x
    y = r.double()
    if normalize:
        y = y / torch.sqrt(y.pow(2).mean(1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    G = group or y.shape[1]
    scale = torch.stack([p.abs().amax(1) / 448 for p in y.split(G, 1)], 1)
    return r, y, scale, scale.repeat_interleave(G, 1)[:, :y.shape[1]]


def check_norm(x, add, w, eps, group, normalize, q, scale, resid):
    r, y, s, per = norm_ref(x, add, w, eps, group, normalize)
    if resid is not None:
        assert torch.equal(resid, r)
    # a thread adds at most 64 squares in turn, then ten joining steps: 75 roundings of the
    # sum, halved by the root, and a dozen around it
    rel = 64 * U
    within(scale, s, rel * s, "scale")
    v = torch.where(per > 0, y / per.clamp_min(1e-300), torch.zeros_like(y))
    tol = torch.clamp(v.abs() * 2 ** -4, min=2 ** -10) + 4 * rel * v.abs()
    within(q.float(), v, tol * (1 + 2 ** -20), "codes")


@pytest.mark.parametrize("dtype", [TB, TH, T32])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 6144), (3, 7), (5, 33), (2, 64), (9, 255), (3, 34), (5, 254), (2, 514), (310, 2052), (300, 256),
                                 (7, 520), (5, 1000), (4, 1024), (700, 1032), (3, 2050),
                                 (400, 4096), (2, 8200), (310, 8200), (2, 16384), (310, 16384),
                                 (3, 16392), (2, 32768), (310, 32768), (2, 32767)])
def test_norm_matches_its_formula(T, H, dtype):
    x, add = randn(1, T, H, dtype=dtype, scale=2), randn(2, T, H, dtype=dtype)
    w = (1 + 0.2 * randn(3, H)).to(dtype)
    for group, a, wt, nrm in [(0, add, w, True), (32, add, None, True), (128, None, w, True),
                              (64, None, None, False), (256, add, w, True), (0, None, w, False)]:
        q = torch.empty(T, H, dtype=F8, device="cuda")
        n = -(-H // group) if group else 1
        scale = torch.empty(T, n, device="cuda")
        resid = torch.empty_like(x)
        moe.moe_rmsnorm_e4m3(x, q, scale, add=a, weight=wt, resid=resid, eps=1e-6, group=group,
                             normalize=nrm)
        check_norm(x, a, wt, 1e-6, group, nrm, q, scale, resid)


@pytest.mark.parametrize("off,pad", [(0, 8), (8, 24), (1, 7), (3, 0)])
def test_norm_strides_and_in_place_residual(off, pad):
    T, H = 17, 640
    big = randn(4, T, off + H + pad, dtype=TB)
    x = big[:, off:off + H]
    add = randn(5, T, H, dtype=TB)
    qb = torch.zeros(T, H + pad + off, dtype=F8, device="cuda")
    q = qb[:, off:off + H]
    scale = torch.empty(T, 1, device="cuda")
    x0, guard = x.clone(), big.clone()
    moe.moe_rmsnorm_e4m3(x, q, scale, add=add, resid=x)
    check_norm(x0, add, None, 1e-6, 0, True, q, scale, x)
    guard[:, off:off + H] = x
    assert torch.equal(big, guard)  # nothing outside the rows was written
    rest = torch.cat([qb[:, :off], qb[:, off + H:]], 1).float()
    assert not bool(rest.any())
    add2 = add.clone()
    moe.moe_rmsnorm_e4m3(x0, q, scale, add=add2, resid=add2)
    check_norm(x0, add, None, 1e-6, 0, True, q, scale, add2)


def test_norm_zero_tiny_and_special_rows():
    H = 256
    x = randn(6, 8, H)
    x[0] = 0
    x[1] = 2.0 ** -120
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] *= 1e15
    x[5] = 2.0 ** -99
    x[6, 1:] = 0
    q, s = torch.empty(8, H, dtype=F8, device="cuda"), torch.empty(8, 1, device="cuda")
    moe.moe_rmsnorm_e4m3(x, q, s, normalize=False)
    assert float(s[0]) == 0 and float(s[1]) == 0 and not bool(q[:2].float().any())
    assert math.isnan(float(s[2])) and bool(torch.isnan(q[2].float()).all())
    assert not math.isfinite(float(s[3]))
    ok = [4, 5, 6, 7]
    check_norm(x[ok], None, None, 0, 0, False, q[ok], s[ok], None)
    moe.moe_rmsnorm_e4m3(x, q, s)
    assert float(s[0]) == 0 and not bool(q[0].float().any())
    assert math.isnan(float(s[2])) and not math.isfinite(float(s[3]))
    check_norm(x[[4, 6, 7]], None, None, 1e-6, 0, True, q[[4, 6, 7]], s[[4, 6, 7]], None)


# ------------------------------------------------------------------- sorting, rows, back
def make_ids(seed, T, k, E, drop=0.0):
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, size=(T, k)).astype(np.int32)
    if drop:
        ids[g.random((T, k)) < drop] = -1
    return ids


def sort_ref(ids, E):
    flat = ids.reshape(-1).astype(np.int64)
    live = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(live, flat, E), kind="stable")
    n = int(live.sum())
    perm = np.full(flat.size, -1, np.int32)
    perm[:n] = order[:n]
    pos = np.full(flat.size, -1, np.int32)
    pos[order[:n]] = np.arange(n)
    off = np.zeros(E + 1, np.int32)
    off[1:] = np.cumsum(np.bincount(flat[live], minlength=E))
    return off, perm, pos.reshape(ids.shape)


def sort_gpu(ids, E):
    d = torch.from_numpy(ids).cuda()
    T, k = ids.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    off, perm = torch.full((E + 1,), 77, **i32), torch.full((T * k,), 77, **i32)
    pos = torch.full((T, k), 77, **i32)
    moe.moe_sort_tokens(d, E, off, perm, pos)
    return off, perm, pos


@pytest.mark.parametrize("T,k,E", [(0, 3, 5), (1, 1, 1), (1, 8, 256), (3, 2, 8), (16, 8, 256),
                                   (31, 1, 2), (257, 8, 256), (256, 8, 33), (300, 7, 31),
                                   (2049, 1, 4), (8192, 8, 256), (65535, 16, 100)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_sort_is_stable_and_complete(T, k, E, drop):
    ids = make_ids(T + k, T, k, E, drop)
    if drop and T:  # ids past the experts are dropped as well
        ids.reshape(-1)[::5] = E
        ids.reshape(-1)[::7] = 2 ** 31 - 1
    for got, want in zip(sort_gpu(ids, E), sort_ref(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T,k,E,H,dtype,S", [
    (1, 1, 1, 1, TB, 0), (1, 8, 256, 6144, F8, 1), (5, 2, 8, 33, TB, 0), (16, 8, 256, 6144, F8, 48),
    (7, 3, 9, 77, F8, 3), (33, 16, 64, 130, TH, 0), (200, 4, 16, 2050, TB, 0),
    (3, 2, 4, 16384, T32, 1), (3000, 8, 256, 512, TB, 0), (9, 2, 4, 30001, F8, 1)])
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
def test_dispatch_moves_rows_and_scales(T, k, E, H, dtype, S, drop):
    ids = make_ids(3, T, k, E, drop)
    off, perm, pos = sort_gpu(ids, E)
    pad = 16 if H % 16 == 0 else 0
    raw = randn(7, T, H + pad).to(dtype)
    x = raw[:, :H]
    xs = torch.full((T * k, H), 1.0, device="cuda").to(dtype)
    sc = randn(8, T, S) if S else None
    scs = torch.full((T * k, S), 7.0, device="cuda") if S else None
    moe.moe_dispatch_rows(x, pos, off, xs, scale=sc, scale_s=scs)
    p = perm.long()
    live = p >= 0
    want = torch.zeros(T * k, H, device="cuda")
    want[live] = x.float()[p[live] // k]
    assert torch.equal(xs.float(), want)
    if S:
        ws = torch.zeros(T * k, S, device="cuda")
        ws[live] = sc[p[live] // k]
        assert torch.equal(scs, ws)


def combine_ref(y, pos, w, add, H):
    """(sum, sum of |terms|) in 64 bits."""
    T, k = pos.shape
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    if add is not None:
        out += add.double()
        mag += add.double().abs()
    for j in range(k):
        live = pos[:, j] >= 0
        term = y[pos[live, j].long()].double()
        if w is not None:
            term = term * w[live, j, None].double()
        out[live] += term
        mag[live] += term.abs()
    return out, mag


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (1, 8, 256, 6144), (5, 2, 8, 33), (7, 3, 8, 34),
                                     (90, 4, 8, 518), (33, 16, 64, 136), (64, 9, 40, 520), (200, 4, 16, 2050),
                                     (1031, 2, 8, 4096)])
@pytest.mark.parametrize("dt,od", [(T32, T32), (TB, TB), (TB, T32), (TH, TH), (TH, T32)])
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
def test_combine_and_its_gradients(T, k, E, H, dt, od, drop):
    ids = make_ids(5, T, k, E, drop)
    off, perm, pos = sort_gpu(ids, E)
    live = perm >= 0
    y = randn(9, T * k, H, dtype=dt)
    y[~live] = float("nan")  # rows of no slot are never read
    w = randn(10, T, k)
    w[pos < 0] = float("nan")
    add = randn(11, T, H, dtype=od)
    for ww, aa in [(w, add), (None, None), (w, None)]:
        out = torch.empty(T, H, dtype=od, device="cuda")
        moe.moe_combine_rows(y, pos, out, w=ww, add=aa)
        ref, mag = combine_ref(y, pos, ww, aa, H)
        # one rounding a term (fused multiply-add) and one of the result
        within(out, ref, (k + 1) * U * mag + half_step(od) * ref.abs() * (1 + 2 ** -7) + 1e-7 *
               (od == TH), "combine")
        if aa is not None:  # in place
            aa2 = aa.clone()
            moe.moe_combine_rows(y, pos, aa2, w=ww, add=aa2)
            assert torch.equal(aa2, out)
    if od != dt:
        return
    dout = randn(12, T, H, dtype=dt)
    dy = torch.full_like(y, 3.0)
    dw = torch.full((T, k), 3.0, device="cuda")
    moe.moe_combine_rows_grad(dout, y, pos, off, w, dy, dw)
    want = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    p = perm[live].long()
    want[live] = dout.double()[p // k] * w.reshape(-1)[p, None].double()
    within(dy, want, (U + half_step(dt)) * (1 + 2 ** -7) * want.abs() + 1e-7 * (dt == TH), "dy")
    assert not bool(dy[~live].float().any())
    ref = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    prod = dout.double()[p // k] * y[live].double()
    ref[p], mag[p] = prod.sum(1), prod.abs().sum(1)
    # a thread's fused sum, five joining steps in a warp and up to eight warps
    steps = 8 * -(-H // 2048) + 8 + 5 + 8
    within(dw.reshape(-1), ref, steps * U * mag, "dw")
    dx = torch.empty(T, H, dtype=dt, device="cuda")
    moe.moe_dispatch_rows_grad(dy, pos, dx)
    ref, mag = combine_ref(dy, pos, None, None, H)
    within(dx, ref, k * U * mag + half_step(dt) * ref.abs() * (1 + 2 ** -7) + 1e-7 * (dt == TH),
           "dx")


def test_gradients_against_differences():
    """The operators are linear in each operand, so a difference over a whole step is exact."""
    T, k, E, H = 11, 3, 6, 72
    ids = make_ids(6, T, k, E, 0.2)
    off, perm, pos = sort_gpu(ids, E)
    y, w = randn(13, T * k, H), randn(14, T, k)
    w[pos < 0] = 0
    dout, dirs = randn(15, T, H), (randn(16, T * k, H), randn(17, T, k))
    dirs[1][pos < 0] = 0

    def f(yy, ww):
        out = torch.empty(T, H, device="cuda")
        moe.moe_combine_rows(yy, pos, out, w=ww)
        return (out.double() * dout.double()).sum()

    dy, dw = torch.empty_like(y), torch.empty_like(w)
    moe.moe_combine_rows_grad(dout, y, pos, off, w, dy, dw)
    base = float(f(y, w))
    tol = 64 * U * T * H * 4  # roundings of a few units in each of T * H terms
    assert abs(float(f(y + dirs[0], w)) - base - float((dy.double() * dirs[0]).sum())) < tol
    assert abs(float(f(y, w + dirs[1])) - base - float((dw.double() * dirs[1]).sum())) < tol
    # rows out and their gradient back: <dispatch(x), g> = <x, dispatch_grad(g)>
    x, g = randn(18, T, H), randn(19, T * k, H)
    xs, dx = torch.empty_like(g), torch.empty_like(x)
    moe.moe_dispatch_rows(x, pos, off, xs)
    moe.moe_dispatch_rows_grad(g, pos, dx)
    assert abs(float((xs.double() * g).sum() - (dx.double() * x).sum())) < tol


@pytest.mark.parametrize("H,dtype", [(8, TB), (9, TB), (64, T32)])
def test_most_tokens_and_slots(H, dtype):
    """65535 tokens with 16 slots each: rows out and back with weights of 1/16 are the tokens."""
    T, k, E = 65535, 16, 256
    off, perm, pos = sort_gpu(make_ids(8, T, k, E), E)
    x = randn(1, T, H).to(dtype)
    xs = torch.empty(T * k, H, dtype=dtype, device="cuda")
    moe.moe_dispatch_rows(x, pos, off, xs)
    out = torch.empty_like(x)
    moe.moe_combine_rows(xs, pos, out, w=torch.full((T, k), 1 / 16, device="cuda"))
    # sixteen equal terms: with 8 bits of significand every partial sum is exact in fp32; a term
    # of 24 bits is not (three of them need 26), and each of its sums rounds once
    few = torch.finfo(dtype).eps > 2 ** -20
    within(out, x.double(), 0 if few else k * U * x.double().abs(), "back")
    dx = torch.empty_like(x)
    moe.moe_dispatch_rows_grad(xs, pos, dx)
    within(dx, 16 * x.double(), 0 if few else k * U * 16 * x.double().abs(), "dx")
    dy, dw = torch.empty_like(xs), torch.empty(T, k, device="cuda")
    moe.moe_combine_rows_grad(x, xs, pos, off, None, dy, dw)
    assert torch.equal(dy, xs)
    sq = (x.double() ** 2).sum(1, keepdim=True)
    within(dw, sq.expand(T, k), (8 + 16) * U * sq, "dw")


# ------------------------------------------------------------------------------ linear
def rows8(v):
    s = v.abs().amax(-1) / 448
    return (v / s[..., None]).to(F8), s.contiguous()


def linear_ref(x, w, xs, ws, bias, act, res, offsets, N):
    """(value, bound on the accumulated error before the output's rounding) in 64 bits."""
    R, K = x.shape
    out = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(out)
    w3 = w if offsets is not None else w[None]
    ends = offsets if offsets is not None else [0, R]
    # the tensor cores add 16 (or 32) products at a time, each sum truncated to fp32 or less:
    # K / 16 steps of 2^-23 of the magnitudes, as much again inside them, and the epilogue
    steps = (K / 8 + 16) * 2 * U
    for e in range(w3.shape[0]):
        a, b = ends[e], ends[e + 1]
        if b <= a:
            continue
        xd, wd = x[a:b].double(), w3[e].double()
        z, m = xd @ wd.t(), xd.abs() @ wd.abs().t()
        if ws is not None:
            f = (ws[e] if offsets is not None else ws).double()
            z, m = z * f, m * f.abs()
        if xs is not None:
            z, m = z * xs[a:b, None].double(), m * xs[a:b, None].double().abs()
        if bias is not None:
            bb = (bias[e] if offsets is not None else bias).double()
            z, m = z + bb, m + bb.abs()
        d = steps * m
        if act == "relu":
            z = z.clamp_min(0)
        elif act == "silu":
            z, d = z * torch.sigmoid(z), 1.1 * d
        elif act == "gelu":
            z, d = z * 0.5 * torch.erfc(-z * math.sqrt(0.5)), 1.13 * d + 4 * U * z.abs()
        elif act == "swiglu":
            g, u = z[:, :N], z[:, N:]
            dg, du = d[:, :N], d[:, N:]
            s = g * torch.sigmoid(g)
            z, d = s * u, 1.1 * dg * (u.abs() + du) + s.abs() * du
        if act not in ("none", "relu"):
            d = d + 16 * U * z.abs()
        out[a:b], err[a:b] = z, d
    if res is not None:
        out += res.double()
        err += U * out.abs()
    return out, err


def run_linear(R, N, K, E, dt, od, act, bias, residual, seed=0, counts=None, pad=0, lead=0,
               tail=0):
    rows = 2 * N if act == "swiglu" else N
    es = 1 if dt == F8 else 2
    padx = (pad * 16) // es
    ne = max(1, E)
    xv, wv = randn(seed + 1, R, K), randn(seed + 2, ne, rows, K) / math.sqrt(K)
    xs = ws = None
    if dt == F8:
        (xq, xs), (wq, ws) = rows8(xv), rows8(wv)
    else:
        xq, wq = xv.to(dt), wv.to(dt)
    xb = torch.zeros(R, K + padx, device="cuda").to(dt)
    xb.view(torch.uint8)[:, :K * es] = xq.view(torch.uint8)
    x = xb[:, :K]
    b = randn(seed + 3, ne, rows) if bias else None
    offsets = host = None
    if E:
        if counts is None:
            g = np.random.default_rng(seed)
            counts = g.multinomial(R - lead - tail, g.dirichlet(np.ones(E) * 0.7))
        host = (lead + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
        offsets = torch.from_numpy(host).cuda()
        host = host.tolist()
    else:
        wq, ws = wq[0], ws[0] if ws is not None else None
        b = b[0] if bias else None
    ob = torch.full((R, N + pad), 5.0, dtype=od, device="cuda")
    out = ob[:, :N]
    res = randn(seed + 4, R, N, dtype=od) if residual else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_linear(x, wq, out, x_scale=xs, w_scale=ws, bias=b, act=act, residual=res,
                   offsets=offsets, status=status)
    ref, err = linear_ref(x, wq, xs, ws, b, act, res, host, N)
    if E and res is not None:  # rows of no expert are zero, without the residual
        ref[:host[0]] = 0
        ref[host[-1]:] = 0
    assert int(status) == 0
    within(out, ref, err + half_step(od) * (1 + 2 ** -7) * (ref.abs() + err) + 1e-7 * (od == TH),
           "linear")
    if pad:
        assert bool((ob[:, N:] == 5.0).all())
    return out


@pytest.mark.parametrize("dt", [F8, TB, TH])
@pytest.mark.parametrize("R,N,K", [(1, 1, 16), (1, 128, 128), (2, 129, 144), (15, 8, 64),
                                   (16, 127, 256), (17, 200, 48), (31, 384, 1024), (64, 100, 512),
                                   (65, 256, 80), (255, 130, 336), (256, 128, 2048),
                                   (257, 1000, 128), (1000, 520, 656)])
def test_linear_dense_sizes(R, N, K, dt):
    run_linear(R, N, K, 0, dt, TB, "none", True, True)


@pytest.mark.parametrize("dt", [F8, TB, TH])
@pytest.mark.parametrize("od", [T32, TB, TH])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, True)])
def test_linear_types_and_activations(dt, od, act, bias, residual):
    run_linear(37, 144, 272, 0, dt, od, act, bias, residual, pad=3)
    run_linear(37, 144, 272, 5, dt, od, act, bias, residual, pad=8)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("dt", [F8, TB])
@pytest.mark.parametrize("R,N,K,E", [(1, 64, 64, 1), (1, 64, 64, 256), (8, 256, 512, 64),
                                     (128, 272, 1040, 64), (300, 16, 48, 3), (1500, 144, 528, 7),
                                     (3000, 1040, 1024, 8)])
def test_linear_by_expert(R, N, K, E, dt, act):
    run_linear(R, N, K, E, dt, TB, act, True, False, seed=R)


# sizes at which pairs of CTAs share a tile (the first five) and clusters split K (the others)
@pytest.mark.parametrize("R,N,K,E", [(2100, 1001, 1000, 0), (5000, 1001, 2048, 0),
                                     (6000, 1501, 1024, 0), (2000, 300, 1024, 5),
                                     (3000, 1040, 2000, 8), (257, 1000, 2048, 0),
                                     (130, 700, 3840, 0), (40, 256, 1024, 16),
                                     (256, 128, 4096, 0)])
@pytest.mark.parametrize("od,act,bias,residual", [(TB, "none", True, True), (T32, "silu", True, False),
                                                  (TH, "gelu", False, False),
                                                  (T32, "swiglu", True, True),
                                                  (TB, "swiglu", True, False)])
def test_linear_pairs_and_splits(R, N, K, E, od, act, bias, residual):
    N, K = (N - N % 16 if act == "swiglu" else N), K // 16 * 16
    run_linear(R, N, K, E, F8, od, act, bias, residual, seed=R, pad=5)
    run_linear(R, N, K // 32 * 16, E, TB, od, act, bias, residual, seed=R)


@pytest.mark.parametrize("R,N,K,E", [(300000, 64, 64, 0), (200003, 48, 80, 3), (5, 40000, 64, 0),
                                     (70, 20000, 48, 2)])
def test_linear_many_rows_or_features(R, N, K, E):
    run_linear(R, N, K, E, F8, TB, "none", True, False, seed=3)


@pytest.mark.parametrize("dt", [F8, TB, TH])
@pytest.mark.parametrize("R,N,K,act", [(1, 256, 14336, "none"), (300, 512, 14336, "none"),
                                       (700, 256, 6144, "swiglu"), (3000, 512, 4096, "none")])
def test_linear_fp32_outputs_are_summed_in_fp32(R, N, K, act, dt):
    """An fp32 output is nearer to the exact product than the tensor cores' truncated sums are.

    Sums of 16 MMAs (4 k-blocks), each truncating by at most 2^-23 of what it holds, on the mean
    half of that and half of them past the middle: 16 * 2^-25 = 5e-7 of the result, twice that for
    a product of two; the whole K in tensor memory would lose K / 256 times as much."""
    rows = 2 * N if act == "swiglu" else N
    xv, wv = randn(1, R, K), randn(2, rows, K) / math.sqrt(K)
    xs = ws = None
    if dt == F8:
        (x, xs), (w, ws) = rows8(xv), rows8(wv)
    else:
        x, w = xv.to(dt), wv.to(dt)
    out = torch.empty(R, N, device="cuda")
    moe.moe_linear(x, w, out, x_scale=xs, w_scale=ws, act=act)
    ref, _ = linear_ref(x, w, xs, ws, None, act, None, None, N)
    rel = float((out.double() - ref).norm() / ref.norm())
    assert rel < (2 if act == "swiglu" else 1) * 16 * 2 ** -25 + 4 * U


@pytest.mark.parametrize("counts", [[0, 0, 5, 0], [256, 0, 0, 1], [255, 1, 257, 0], [0, 0, 0, 0],
                                    [16, 16, 16, 16], [1, 511, 17, 33]])
@pytest.mark.parametrize("lead,tail", [(0, 0), (3, 40)])
def test_linear_empty_experts_and_rows_of_no_expert(counts, lead, tail):
    R = lead + sum(counts) + tail
    if R == 0:
        return
    for act in ("none", "swiglu"):
        run_linear(R, 80, 192, 4, F8, TB, act, True, True, counts=counts, lead=lead, tail=tail)


def test_linear_clamps_offsets_to_the_rows():
    """Offsets out of range or out of order never lead out of x: they are read as the running
    maximum of their values clamped to [0, R]."""
    R, N, K, E = 40, 64, 64, 4
    x, w = randn(1, R, K, dtype=TB), randn(2, E, N, K, dtype=TB)
    out = torch.full((R, N), 9.0, device="cuda")
    off = torch.tensor([-7, 10, 4, 2 ** 31 - 1, 30], dtype=torch.int32, device="cuda")
    moe.moe_linear(x, w, out, offsets=off)
    ref, err = linear_ref(x, w, None, None, None, "none", None, [0, 10, 10, 40, 40], N)
    within(out, ref, err + U * ref.abs(), "clamped")


def test_linear_nan_stays_in_its_rows():
    R, N, K = 70, 96, 128
    x, w = randn(1, R, K, dtype=TB), randn(2, N, K, dtype=TB)
    clean = torch.empty(R, N, device="cuda")
    moe.moe_linear(x, w, clean)
    x[3, 5] = float("nan")
    x[64, 1] = float("inf")
    out = torch.empty_like(clean)
    moe.moe_linear(x, w, out, act="relu")
    assert bool(torch.isnan(out[3]).all())
    keep = [r for r in range(R) if r not in (3, 64)]
    assert torch.equal(out[keep], clean[keep].clamp_min(0))


def test_linear_large_offsets_in_weights():
    """Weights past 2^31 elements: the last expert's rows."""
    E, N, K = 40, 4096, 14336
    w = torch.zeros(E, N, K, dtype=F8, device="cuda")
    w[E - 1] = rows8(randn(2, N, K))[0]
    x, xs = rows8(randn(3, 5, K))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = 5
    out = torch.empty(5, N, device="cuda")
    moe.moe_linear(x, w, out, x_scale=xs, offsets=off)
    ref, err = linear_ref(x, w[E - 1], xs, None, None, "none", None, None, N)
    within(out, ref, err + U * ref.abs(), "last expert")


def test_refusals_raise_the_status():
    """What the C entry points refuse reaches Python as MoEError with the status."""
    ids = torch.zeros(3, 17, dtype=torch.int32, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    perm = torch.zeros(51, dtype=torch.int32, device="cuda")
    x, q = randn(1, 4, 72, dtype=TB), torch.empty(4, 72, dtype=F8, device="cuda")
    calls = [lambda: moe.moe_sort_tokens(ids, 4, off, perm, ids),
             lambda: moe.moe_rmsnorm_e4m3(x, q, torch.empty(4, 5, device="cuda"), group=16),
             lambda: moe.moe_linear(x, randn(2, 8, 72, dtype=TB), torch.empty(4, 8, device="cuda"))]
    for f in calls:
        with pytest.raises(moe.MoEError) as e:
            f()
        assert e.value.status == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(ValueError):  # an operand on the host
        moe.moe_rmsnorm_e4m3(x, q, torch.empty(4, 1))


# ------------------------------------------------------------------ together, captured
def test_chain_repeats_bit_for_bit_on_a_stream_and_in_a_graph():
    """Norm -> sort -> rows out -> gate/up -> quantise -> down -> back, eagerly on a side
    stream and as a captured graph: the same bits."""
    T, k, E, H, I = 50, 4, 16, 512, 256
    x, add = randn(1, T, H, dtype=TB), randn(2, T, H, dtype=TB)
    ids = torch.from_numpy(make_ids(1, T, k, E, 0.1)).cuda()
    w = torch.softmax(randn(3, T, k), 1)
    (w1, s1), (w2, s2) = rows8(randn(4, E, 2 * I, H)), rows8(randn(5, E, H, I))
    n, d = T * k, dict(device="cuda")
    i32 = dict(dtype=torch.int32, **d)
    q, sc = torch.empty(T, H, dtype=F8, **d), torch.empty(T, 1, **d)
    r, out = torch.empty_like(x), torch.empty(T, H, dtype=TB, **d)
    off, perm, pos = torch.empty(E + 1, **i32), torch.empty(n, **i32), torch.empty(T, k, **i32)
    xs, xsc = torch.empty(n, H, dtype=F8, **d), torch.empty(n, 1, **d)
    h, y = torch.empty(n, I, dtype=TB, **d), torch.empty(n, H, dtype=TB, **d)
    hq, hs = torch.empty(n, I, dtype=F8, **d), torch.empty(n, 1, **d)

    def chain():
        moe.moe_rmsnorm_e4m3(x, q, sc, add=add, resid=r)
        moe.moe_sort_tokens(ids, E, off, perm, pos)
        moe.moe_dispatch_rows(q, pos, off, xs, scale=sc, scale_s=xsc)
        moe.moe_linear(xs, w1, h, x_scale=xsc, w_scale=s1, act="swiglu", offsets=off)
        moe.moe_rmsnorm_e4m3(h, hq, hs, normalize=False)
        moe.moe_linear(hq, w2, y, x_scale=hs, w_scale=s2, offsets=off)
        moe.moe_combine_rows(y, pos, out, w=w, add=r)

    chain()
    torch.cuda.synchronize()
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            chain()
    side.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for t in (out, y, h, xs, q, hq):
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_linear_on_two_streams_at_once():
    """Calls of every form overlapping on two streams give the bits they give alone."""
    shapes = [(1, 2048, 6144, 0, TB, "silu"), (16, 512, 1024, 0, F8, "none"),
              (200, 1024, 2048, 0, TB, "none"), (1000, 1024, 512, 0, F8, "swiglu"),
              (40, 256, 512, 16, F8, "swiglu"), (3000, 512, 1024, 4, TB, "none")]
    calls = []
    for i, (R, N, K, E, dt, act) in enumerate(shapes):
        rows = 2 * N if act == "swiglu" else N
        x, w = randn(i, R, K).to(dt), randn(i + 50, max(1, E), rows, K).to(dt)
        off = None
        if E:
            off = torch.linspace(0, R, E + 1, device="cuda").int()
        out = torch.empty(R, N, dtype=TB, device="cuda")
        kw = dict(act=act, offsets=off)
        moe.moe_linear(x, w if E else w[0], out, **kw)
        calls.append((x, w if E else w[0], out.clone(), torch.empty_like(out),
                      torch.empty_like(out), kw))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, st in enumerate(streams):
            for x, w, _, o1, o2, kw in (calls if s == 0 else calls[::-1]):
                moe.moe_linear(x, w, o1 if s == 0 else o2, stream=st, **kw)
    torch.cuda.synchronize()
    for _, _, want, o1, o2, _ in calls:
        assert torch.equal(o1, want) and torch.equal(o2, want)


def test_operators_follow_each_other_without_waiting():
    """Each kernel may start while the one before it ends: weights and rows written by the call
    just before are the ones that are read."""
    R, N, K = 64, 256, 512
    src = [randn(i, N, K) for i in range(6)]
    x = randn(9, R, K)
    q, s = torch.empty(N, K, dtype=F8, device="cuda"), torch.empty(N, 1, device="cuda")
    xq, xs = torch.empty(R, K, dtype=F8, device="cuda"), torch.empty(R, 1, device="cuda")
    outs = [torch.empty(R, N, device="cuda") for _ in src]
    moe.moe_rmsnorm_e4m3(x, xq, xs, normalize=False)
    for w, out in zip(src, outs):
        moe.moe_rmsnorm_e4m3(w, q, s, normalize=False)
        moe.moe_linear(xq, q, out, x_scale=xs, w_scale=s[:, 0])
    torch.cuda.synchronize()
    for w, out in zip(src, outs):
        moe.moe_rmsnorm_e4m3(w, q, s, normalize=False)
        torch.cuda.synchronize()
        alone = torch.empty_like(out)
        moe.moe_linear(xq, q, alone, x_scale=xs, w_scale=s[:, 0])
        torch.cuda.synchronize()
        assert torch.equal(out, alone)
