"""A MoE layer whose experts are e4m3 weights with row scales, on the token operators.

The packed layer (`moe_layer_forward`) takes integer experts; this is the routed part of such a
layer (no shared expert) for experts that are kept as 8-bit floating-point rows:

    r   = resid + add                                   (the residual stream, in its own type)
    x   = RMSNorm(r) * norm_weight as e4m3 rows with a scale each
    h   = silu(x_s Wg_e^T) * (x_s Wu_e^T) on the rows sorted by expert, again as e4m3 rows
    out = r + sum_j w[t, j] * (h Wd_e^T)[row of (t, j)]

The experts and weights of each token come from outside: from moe_route_topk, or any other router.
A router wants the normalised hidden states in fp32 or bf16 before forward() runs, which the caller
computes (x here is 8-bit rows and scales only).

Every step runs in the library's kernels on buffers that this object owns, so that a step can
be captured in a CUDA graph.  What the device finds out on the way (a bounded wait that gave up:
the output is then undefined) stays in a status word until read_status() takes it.
"""
from __future__ import annotations

import torch

from . import MOE_OK
from .tokens import (moe_combine_rows, moe_dispatch_rows, moe_linear, moe_rmsnorm_e4m3,
                     moe_sort_tokens)

E4M3 = torch.float8_e4m3fn


def quantize_e4m3(w):
    """w [..., n] (fp32, bf16 or fp16) -> e4m3 codes of the same shape and fp32 scales [...]."""
    rows = w.reshape(-1, w.shape[-1])
    q = torch.empty(rows.shape, dtype=E4M3, device=w.device)
    scale = torch.empty((rows.shape[0], 1), dtype=torch.float32, device=w.device)
    moe_rmsnorm_e4m3(rows, q, scale, normalize=False)
    return q.view(w.shape), scale.view(w.shape[:-1])


class E4m3Experts:
    """Experts of one layer for up to t_max tokens with top_k slots each.

    gate_up [E, 2I, H] (gate rows first) and down [E, H, I] are e4m3 codes with scales
    [E, 2I] and [E, H] (see quantize_e4m3)."""

    def __init__(self, gate_up, gate_up_scale, down, down_scale, top_k, t_max, norm_weight=None,
                 eps=1e-6, dtype=torch.bfloat16):
        E, I2, H = gate_up.shape
        if down.shape != (E, H, I2 // 2) or I2 % 2:
            raise ValueError("gate_up must be [E, 2I, H] and down [E, H, I]")
        self.w1, self.s1, self.w2, self.s2 = gate_up, gate_up_scale, down, down_scale
        self.E, self.I, self.H, self.k, self.t_max = E, I2 // 2, H, top_k, t_max
        self.norm_weight, self.eps, self.dtype = norm_weight, eps, dtype
        n, on = t_max * top_k, {"device": gate_up.device}
        i32, f32 = {"dtype": torch.int32, **on}, {"dtype": torch.float32, **on}
        self.resid = torch.empty((t_max, H), dtype=dtype, **on)
        self.out = torch.empty((t_max, H), dtype=dtype, **on)
        self.q, self.qs = torch.empty((t_max, H), dtype=E4M3, **on), torch.empty((t_max, 1), **f32)
        self.offsets = torch.empty(E + 1, **i32)
        self.perm, self.slot_pos = torch.empty(n, **i32), torch.empty((t_max, top_k), **i32)
        self.xs, self.xss = torch.empty((n, H), dtype=E4M3, **on), torch.empty((n, 1), **f32)
        self.h = torch.empty((n, self.I), dtype=dtype, **on)
        self.hq, self.hs = torch.empty((n, self.I), dtype=E4M3, **on), torch.empty((n, 1), **f32)
        self.y = torch.empty((n, H), dtype=dtype, **on)
        self.status = torch.zeros(1, **i32)

    def forward(self, resid, add, ids, w):
        """resid [T, H] and add (the attention's output, or None) of the layer's dtype, ids int32
        and w fp32 [T, k] as moe_route_topk writes them (ids outside [0, E) are left out).  Returns the new residual stream, a view
        of the layer's buffer."""
        T = resid.shape[0]
        if T > self.t_max:
            raise ValueError(f"{T} tokens, but the layer has room for {self.t_max}")
        n = T * self.k
        r, q, qs, pos = self.resid[:T], self.q[:T], self.qs[:T], self.slot_pos[:T]
        xs, xss, h, y = self.xs[:n], self.xss[:n], self.h[:n], self.y[:n]
        hq, hs, out = self.hq[:n], self.hs[:n], self.out[:T]
        moe_rmsnorm_e4m3(resid, q, qs, add=add, weight=self.norm_weight, resid=r, eps=self.eps)
        moe_sort_tokens(ids, self.E, self.offsets, self.perm[:n], pos)
        moe_dispatch_rows(q, pos, self.offsets, xs, scale=qs, scale_s=xss)
        moe_linear(xs, self.w1, h, x_scale=xss, w_scale=self.s1, act="swiglu",
                   offsets=self.offsets, status=self.status)
        moe_rmsnorm_e4m3(h, hq, hs, normalize=False)
        moe_linear(hq, self.w2, y, x_scale=hs, w_scale=self.s2, offsets=self.offsets,
                   status=self.status)
        moe_combine_rows(y, pos, out, w=w, add=r)
        return out

    def read_status(self):
        """The status of the forward calls since the last reading (MOE_OK, or MOE_ERR_TIMEOUT when
        one's output is undefined), cleared by it.  Waits for the current stream."""
        status = int(self.status)
        if status != MOE_OK:
            self.status.zero_()
        return status
