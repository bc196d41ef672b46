"""Token operators: what surrounds the experts in a user's own layers (include/moe.h, last part).

Experts chosen from router logits with the gradient back, RMS norm to e4m3 rows, tokens sorted by
expert and back with gradients, SwiGLU that keeps its input in 8 bits for its gradient, and the
matrix product with its epilogue.  As in the rest of the package every step runs in the library's
kernels, on the operands' device (which need not be the current one) and its current stream or a
given torch.cuda.Stream of that device, into tensors that the caller owns; nothing is allocated and
every call may be captured into a graph.  Shapes, types, strides and devices are checked (the
C entry points see only addresses): a wrong one raises ValueError or TypeError, an error of the
C entry point MoEError.

The calls stand outside autograd, as the rest of the package does: they record no graph, whatever
their operands require, so a model that trains through them makes them in the forward and backward
of a torch.autograd.Function.  What they write counts as written: version counters move on, and an
output that requires a gradient is refused while graphs are recorded.

At decode sizes the host side of a call counts as much as its kernel, so tensors are read and
checked by a small extension module (csrc/tokens_py.cpp) and not through ctypes: 2.3 us for a whole
call of the norm where that took 7.3.
"""
from __future__ import annotations

import torch  # (its libraries are the extension module's)

from . import MOE_OK, MoEError, lib

ROUTERS = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}


def _made_for_this_torch(module):
    """The extension module, unless it was compiled against another torch's headers."""
    made_for = getattr(module, "torch_version", "another version")
    if made_for != str(torch.__version__):
        raise ImportError(f"the token operators' entry points were built for torch "
                          f"{made_for}, this is {torch.__version__}: build again "
                          "(routed_expert_ffn_route_gb300.build())")
    return module


class _Late:
    """Stands for the extension module until the first call, which raises if the library has not
    been built (the two are built together)."""

    def __getattr__(self, name):
        global _native
        lib()
        try:
            from . import _tokens_native
        except ImportError as e:
            raise ImportError("the token operators' entry points have not been built for this "
                              "Python: build() makes them where torch has CUDA and Python's "
                              "headers are installed") from e
        _native = _made_for_this_torch(_tokens_native)
        return getattr(_native, name)


_native = _Late()


def _check(status, where):
    if status != MOE_OK:
        raise MoEError(status, where)


def moe_rmsnorm_e4m3(x, q, scale, add=None, weight=None, resid=None, eps=1e-6, group=0,
                     normalize=True, stream=None):
    """r = x + add -> resid; q (float8_e4m3fn [T, H]) and scale (fp32 [T, ceil(H / group)],
    group 0: one a row) of r * weight / sqrt(mean(r^2) + eps).  normalize=False quantises
    r * weight itself.  x, add, resid [T, H] and weight [H] of one type, rows may lie apart."""
    _check(_native.rmsnorm(x, q, scale, add, weight, resid, eps, group, normalize,
                           stream), "moe_rmsnorm_e4m3")


def moe_sort_tokens(ids, n_experts, offsets, perm, slot_pos, stream=None):
    """ids int32 [T, k] -> offsets [E + 1], perm [T * k], slot_pos [T, k], all int32."""
    _check(_native.sort(ids, n_experts, offsets, perm, slot_pos, stream),
           "moe_sort_tokens")


def moe_dispatch_rows(x, slot_pos, offsets, xs, scale=None, scale_s=None, stream=None):
    """xs[slot_pos[t, j]] = x[t] ([T * k, H], the rest zero); scale [T, S] -> scale_s alike."""
    _check(_native.dispatch(x, slot_pos, offsets, xs, scale, scale_s, stream),
           "moe_dispatch_rows")


def moe_combine_rows(y, slot_pos, out, w=None, add=None, stream=None):
    """out[t] = add[t] + sum_j w[t, j] * y[slot_pos[t, j]] (slots of -1 left out)."""
    _check(_native.combine(y, slot_pos, out, w, add, stream), "moe_combine_rows")


def moe_combine_rows_grad(dout, y, slot_pos, offsets, w, dy, dw, stream=None):
    """dy[slot_pos[t, j]] = w[t, j] * dout[t] (the rest zero), dw[t, j] = <dout[t], y[slot]>."""
    _check(_native.combine_grad(dout, y, slot_pos, offsets, w, dy, dw, stream),
           "moe_combine_rows_grad")


def moe_dispatch_rows_grad(dxs, slot_pos, dx, stream=None):
    """dx[t] = sum_j dxs[slot_pos[t, j]] (slots of -1 left out)."""
    _check(_native.dispatch_grad(dxs, slot_pos, dx, stream), "moe_dispatch_rows_grad")


def _router(router):
    code = ROUTERS.get(router)
    if code is None:
        raise ValueError(f"router must be one of {sorted(ROUTERS)}, got {router!r}")
    return code


def moe_route_logits(logits, ids, w, bias=None, router="softmax", n_group=1, topk_group=1,
                     group_best=2, norm_topk=True, routed_scaling_factor=1.0, stream=None):
    """The k experts of each token from logits [T, E] (fp32, bf16 or fp16) -> ids int32 and w fp32
    [T, k], best first.  Scores are the logits' softmax or sigmoid, see ROUTERS; bias (fp32 [E]) is
    added for the choice alone.  With n_group > 1 only the topk_group groups whose group_best
    largest scores have the largest sum are chosen from.  An expert whose logit is -inf or NaN is
    not available; a slot that none is left for gets id -1 and weight 0."""
    _check(_native.route_logits(logits, ids, w, bias, _router(router), n_group, topk_group,
                                group_best, norm_topk, routed_scaling_factor, stream),
           "moe_route_logits")


def moe_route_logits_grad(dw, logits, ids, dlogits, router="softmax", norm_topk=True,
                          routed_scaling_factor=1.0, stream=None):
    """dlogits [T, E] of dw [T, k], for the ids that moe_route_logits chose; dlogits is not the logits'
    own memory."""
    _check(_native.route_logits_grad(dw, logits, ids, dlogits, _router(router), norm_topk,
                                     routed_scaling_factor, stream), "moe_route_logits_grad")


def moe_swiglu_e4m3(z, h, q, scale, group=128, stream=None):
    """h [R, I] = silu(z[:, :I]) * z[:, I:], and z itself as q (float8_e4m3fn [R, 2I]) and scale
    (fp32 [R, 2 * ceil(I / group)]: the groups of the first half, then of the second)."""
    _check(_native.swiglu(z, h, q, scale, group, stream), "moe_swiglu_e4m3")


def moe_swiglu_e4m3_grad(dh, q, scale, dz, h=None, group=128, stream=None):
    """dz [R, 2I] of dh [R, I], where z is what q and scale hold; h: the product again."""
    _check(_native.swiglu_grad(dh, q, scale, dz, h, group, stream), "moe_swiglu_e4m3_grad")


def moe_linear(x, w, out, x_scale=None, w_scale=None, bias=None, act="none", residual=None,
               offsets=None, status=None, stream=None):
    """out = act((x w^T) * x_scale * w_scale + bias) + residual; see ACTIVATIONS for act.

    Dense: w [N, K] (SwiGLU: [2N, K], gate rows first).  By expert: w [E, N, K] and offsets
    int32 [E + 1], rows offsets[e] .. offsets[e + 1] of x using expert e; w_scale and bias
    have w's leading dimensions.  x_scale [R] or [R, 1].  x and w are both e4m3, bf16, fp16 or int8
    (codes and scales as moe_quantize_rows makes them)."""
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    _check(_native.linear(x, w, out, x_scale, w_scale, bias, code, residual, offsets, status,
                          stream), "moe_linear")
