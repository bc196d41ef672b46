"""Token operators: what surrounds the experts in a user's own layers (include/moe.h, last part).

RMS norm to e4m3 rows, tokens sorted by expert and back with gradients, and the matrix
product with its epilogue.  As in the rest of the package every step runs in the library's
kernels, on the current stream, into tensors that the caller owns; nothing is allocated and
every call may be captured into a graph.  Shapes, types, strides and devices are checked here
(the C entry points see only addresses): a wrong one raises ValueError or TypeError.

At decode sizes the host side of a call counts as much as its kernel: the checks read each
tensor attribute once, and the arguments go to the C entry points as plain integers through a
small extension module (csrc/tokens_py.c) instead of ctypes (5.3 us for a whole call of the norm
where ctypes took 7.3).
"""
from __future__ import annotations

import torch

from . import MOE_DT_BF16, MOE_DT_E4M3, MOE_DT_F16, MOE_DT_F32, MOE_OK, MoEError, lib


class _Late:
    """Stands for the extension module until the first call, which raises if the library has not
    been built (the two are built together)."""

    def __getattr__(self, name):
        global _native
        lib()
        from . import _tokens_native
        _native = _tokens_native
        return getattr(_native, name)


_native = _Late()

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}
_F32, _I32, _E4M3 = torch.float32, torch.int32, torch.float8_e4m3fn
_DTYPES = {_F32: MOE_DT_F32, torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16,
           _E4M3: MOE_DT_E4M3}


def _row_type(dtype) -> int:
    t = _DTYPES.get(dtype)
    if t is None:
        raise TypeError("rows must be float32, bfloat16, float16 or float8_e4m3fn, "
                        f"got {dtype}")
    return t


# the current stream's handle without building a Stream object, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(dev, stream):
    """The handle of `stream`, or of the current stream of the operands' device."""
    if stream is not None:
        return stream.cuda_stream
    if dev < 0:
        raise ValueError("operands must be on a CUDA device")
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _wrong(t, shape, dtype, dev, name):
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device than the first operand")


def _rows(t, shape, dtype, dev, name):
    """Check a [rows, n] operand, whose rows may lie apart; returns (address, row distance)."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        _wrong(t, shape, dtype, dev, name)
    n = shape[1]
    if t.is_contiguous():
        return t.data_ptr(), n
    ld, step = t.stride()
    if step != 1 and n > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if ld < n:
        if shape[0] > 1:
            raise ValueError(f"{name}'s rows overlap")
        ld = n
    return t.data_ptr(), ld


def _flat(t, shape, dtype, dev, name):
    """Check a contiguous operand; returns its address."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        _wrong(t, shape, dtype, dev, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _check(status, where):
    if status != MOE_OK:
        raise MoEError(status, where)


def moe_rmsnorm_e4m3(x, q, scale, add=None, weight=None, resid=None, eps=1e-6, group=0,
                     normalize=True, stream=None):
    """r = x + add -> resid; q (float8_e4m3fn [T, H]) and scale (fp32 [T, ceil(H / group)],
    group 0: one a row) of r * weight / sqrt(mean(r^2) + eps).  normalize=False quantises
    r * weight itself."""
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    T, H = shape
    px, ldx = _rows(x, shape, dt, dev, "x")
    pq, ldq = _rows(q, shape, _E4M3, dev, "q")
    ps = _flat(scale, (T, -(-H // group) if group > 0 else 1), _F32, dev, "scale")
    pa, lda = (None, 0) if add is None else _rows(add, shape, dt, dev, "add")
    pr, ldr = (None, 0) if resid is None else _rows(resid, shape, dt, dev, "resid")
    pw = None if weight is None else _flat(weight, (H,), dt, dev, "weight")
    _check(_native.rmsnorm(T, H, px, ldx, _row_type(dt), pa, lda, pw, eps,
                           1 if normalize else 0, group, pr, ldr, pq, ldq, ps,
                           _stream_of(dev, stream)), "moe_rmsnorm_e4m3")


def moe_sort_tokens(ids, n_experts, offsets, perm, slot_pos, stream=None):
    """ids int32 [T, k] -> offsets [E + 1], perm [T * k], slot_pos [T, k], all int32."""
    shape, dev = ids.shape, ids.get_device()
    T, k = shape
    pi = _flat(ids, shape, _I32, dev, "ids")
    po = _flat(offsets, (n_experts + 1,), _I32, dev, "offsets")
    pp = _flat(perm, (T * k,), _I32, dev, "perm")
    ps = _flat(slot_pos, shape, _I32, dev, "slot_pos")
    _check(_native.sort(T, k, n_experts, pi, po, pp, ps, _stream_of(dev, stream)),
           "moe_sort_tokens")


def moe_dispatch_rows(x, slot_pos, offsets, xs, scale=None, scale_s=None, stream=None):
    """xs[slot_pos[t, j]] = x[t] ([T * k, H], the rest zero); scale [T, S] -> scale_s alike."""
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    T, H = shape
    k, E1 = slot_pos.shape[1], offsets.numel()
    px, ldx = _rows(x, shape, dt, dev, "x")
    pxs = _flat(xs, (T * k, H), dt, dev, "xs")
    pp = _flat(slot_pos, (T, k), _I32, dev, "slot_pos")
    po = _flat(offsets, (E1,), _I32, dev, "offsets")
    S = ldsc = 0
    psc = pss = None
    if scale is not None:
        S = scale.shape[1]
        psc, ldsc = _rows(scale, (T, S), _F32, dev, "scale")
        if scale_s is None:
            raise ValueError("scale_s is needed with scale")
        pss = _flat(scale_s, (T * k, S), _F32, dev, "scale_s")
    _check(_native.dispatch(T, k, E1 - 1, H, _row_type(dt), px, ldx, pp, po, pxs, S, psc,
                            ldsc, pss, _stream_of(dev, stream)), "moe_dispatch_rows")


def moe_combine_rows(y, slot_pos, out, w=None, add=None, stream=None):
    """out[t] = add[t] + sum_j w[t, j] * y[slot_pos[t, j]] (slots of -1 left out)."""
    T, k = slot_pos.shape
    H, ot, yt, dev = out.shape[1], out.dtype, y.dtype, y.get_device()
    py = _flat(y, (T * k, H), yt, dev, "y")
    pp = _flat(slot_pos, (T, k), _I32, dev, "slot_pos")
    po, ldo = _rows(out, (T, H), ot, dev, "out")
    pa, lda = (None, 0) if add is None else _rows(add, (T, H), ot, dev, "add")
    pw = None if w is None else _flat(w, (T, k), _F32, dev, "w")
    _check(_native.combine(T, k, H, py, _row_type(yt), pp, pw, pa, lda, po, ldo,
                           _row_type(ot), _stream_of(dev, stream)), "moe_combine_rows")


def moe_combine_rows_grad(dout, y, slot_pos, offsets, w, dy, dw, stream=None):
    """dy[slot_pos[t, j]] = w[t, j] * dout[t] (the rest zero), dw[t, j] = <dout[t], y[slot]>."""
    T, k = slot_pos.shape
    H, dt, dev, E1 = dout.shape[1], dout.dtype, dout.get_device(), offsets.numel()
    pd, ldd = _rows(dout, (T, H), dt, dev, "dout")
    py = _flat(y, (T * k, H), dt, dev, "y")
    pdy = _flat(dy, (T * k, H), dt, dev, "dy")
    pdw = _flat(dw, (T, k), _F32, dev, "dw")
    pp = _flat(slot_pos, (T, k), _I32, dev, "slot_pos")
    po = _flat(offsets, (E1,), _I32, dev, "offsets")
    pw = None if w is None else _flat(w, (T, k), _F32, dev, "w")
    _check(_native.combine_grad(T, k, E1 - 1, H, _row_type(dt), pd, ldd, py, pp, po, pw,
                                pdy, pdw, _stream_of(dev, stream)),
           "moe_combine_rows_grad")


def moe_dispatch_rows_grad(dxs, slot_pos, dx, stream=None):
    """dx[t] = sum_j dxs[slot_pos[t, j]] (slots of -1 left out)."""
    T, k = slot_pos.shape
    H, dt, xt, dev = dx.shape[1], dxs.dtype, dx.dtype, dxs.get_device()
    pd = _flat(dxs, (T * k, H), dt, dev, "dxs")
    pp = _flat(slot_pos, (T, k), _I32, dev, "slot_pos")
    px, ldx = _rows(dx, (T, H), xt, dev, "dx")
    _check(_native.dispatch_grad(T, k, H, _row_type(dt), pd, pp, px, ldx, _row_type(xt),
                                 _stream_of(dev, stream)), "moe_dispatch_rows_grad")


def moe_linear(x, w, out, x_scale=None, w_scale=None, bias=None, act="none", residual=None,
               offsets=None, status=None, stream=None):
    """out = act((x w^T) * x_scale * w_scale + bias) + residual; see ACTIVATIONS for act.

    Dense: w [N, K] (SwiGLU: [2N, K], gate rows first).  By expert: w [E, N, K] and offsets
    int32 [E + 1], rows offsets[e] .. offsets[e + 1] of x using expert e; w_scale and bias
    have w's leading dimensions.  x_scale [R] or [R, 1]."""
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    R, K = shape
    N, ot = out.shape[1], out.dtype
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    lead = (2 * N if act == "swiglu" else N,)
    E, po = 0, None
    if offsets is not None:
        E = offsets.numel() - 1
        if E < 1:
            raise ValueError("offsets must hold E + 1 values")
        po = _flat(offsets, (E + 1,), _I32, dev, "offsets")
        lead = (E,) + lead
    px, ldx = _rows(x, shape, dt, dev, "x")
    pw = _flat(w, lead + (K,), dt, dev, "w")
    pout, ldo = _rows(out, (R, N), ot, dev, "out")
    pr, ldr = (None, 0) if residual is None else _rows(residual, (R, N), ot, dev, "residual")
    pxs = None if x_scale is None else _flat(
        x_scale, (R,) if x_scale.dim() == 1 else (R, 1), _F32, dev, "x_scale")
    pws = None if w_scale is None else _flat(w_scale, lead, _F32, dev, "w_scale")
    pb = None if bias is None else _flat(bias, lead, _F32, dev, "bias")
    pst = None if status is None else _flat(status, (1,), _I32, dev, "status")
    _check(_native.linear(R, N, K, E, px, ldx, _row_type(dt), pxs, pw, pws, pb, code, pr, ldr,
                          po, pout, ldo, _row_type(ot), pst, _stream_of(dev, stream)),
           "moe_linear")
