"""PyTorch autograd for the fused attention + JVP: a differentiable
``(o, to) = attn_jvp_autograd(q, k, v, tq, tk, tv)`` whose forward is the C
ABI's ``attn_jvp_fwd_stats`` and whose backward is ``attn_jvp_bwd`` (with
``causal=True``: ``attn_jvp_fwd_causal_stats`` and ``attn_jvp_bwd_causal``), so that
a loss built from both O and its tangent tO (as rCM's consistency-distillation
objective is) back-propagates into Q, K, V and the tangents through the
library's kernels only.  ``softcap``, ``slopes``, ``key_begin``, ``key_end`` and shared
key heads take the scored entry points (``attn_jvp_fwd_scored_stats``,
``attn_jvp_bwd_scored``).  Plumbing: argument marshalling and saved tensors;
every step of the computation runs in the CUDA library.
"""
from __future__ import annotations

import torch

from ._binding import attn_jvp_bwd, attn_jvp_bwd_causal, attn_jvp_fwd_causal_stats, attn_jvp_fwd_stats
from ._scored import attn_jvp_bwd_scored, attn_jvp_fwd_scored_stats, key_bounds

__all__ = ["AttnJvpFunction", "AttnJvpScoredFunction", "attn_jvp_autograd"]


class AttnJvpFunction(torch.autograd.Function):
    """Forward: O and tO (bf16, [B, H, Lq, d]); backward: the six gradients."""

    @staticmethod
    def forward(ctx, q, k, v, tq, tk, tv, scale, causal=False):
        q, k, v, tq, tk, tv = (x.contiguous() for x in (q, k, v, tq, tk, tv))
        fwd = attn_jvp_fwd_causal_stats if causal else attn_jvp_fwd_stats
        o, to, lse, mu = fwd(q, k, v, tq, tk, tv, scale)
        ctx.save_for_backward(q, k, v, tq, tk, tv, o, to, lse, mu)
        ctx.scale = scale
        ctx.causal = causal
        return o, to

    @staticmethod
    def backward(ctx, dout, dtout):
        q, k, v, tq, tk, tv, o, to, lse, mu = ctx.saved_tensors
        # an output that does not reach the loss has no cotangent: zeros
        dout = torch.zeros_like(o) if dout is None else dout.to(o.dtype).contiguous()
        dtout = torch.zeros_like(to) if dtout is None else dtout.to(to.dtype).contiguous()
        bwd = attn_jvp_bwd_causal if ctx.causal else attn_jvp_bwd
        g = bwd(q, k, v, tq, tk, tv, o, to, lse, mu, dout, dtout, ctx.scale)
        return g["dq"], g["dk"], g["dv"], g["dtq"], g["dtk"], g["dtv"], None, None


class AttnJvpScoredFunction(torch.autograd.Function):
    """The same with modified scores and shared key heads; slopes and bounds are
    constants, and the gradients are not differentiable themselves."""

    @staticmethod
    def forward(ctx, q, k, v, tq, tk, tv, scale, softcap, slopes, key_begin, key_end):
        q, k, v, tq, tk, tv = (x.contiguous() for x in (q, k, v, tq, tk, tv))
        o, to, lse, mu = attn_jvp_fwd_scored_stats(q, k, v, tq, tk, tv, scale, softcap, slopes, key_begin, key_end)
        ctx.save_for_backward(q, k, v, tq, tk, tv, o, to, lse, mu, slopes, key_begin, key_end)
        ctx.scale = scale
        ctx.softcap = softcap
        return o, to

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dtout):
        q, k, v, tq, tk, tv, o, to, lse, mu, slopes, key_begin, key_end = ctx.saved_tensors
        dout = torch.zeros_like(o) if dout is None else dout.to(o.dtype).contiguous()
        dtout = torch.zeros_like(to) if dtout is None else dtout.to(to.dtype).contiguous()
        g = attn_jvp_bwd_scored(q, k, v, tq, tk, tv, o, to, lse, mu, dout, dtout, ctx.scale, ctx.softcap, slopes,
                                key_begin, key_end)
        return g["dq"], g["dk"], g["dv"], g["dtq"], g["dtk"], g["dtv"], None, None, None, None, None


def attn_jvp_autograd(q, k, v, tq, tk, tv, scale=None, causal=False, softcap=0.0, slopes=None, key_begin=None,
                      key_end=None):
    """Differentiable (O, tO) for bf16 [B, H, L, 128] CUDA tensors; ``causal``:
    key j visible to query row i iff j <= i + (Lk - Lq).  ``softcap``, ``slopes``,
    ``key_begin`` and ``key_end`` as in ``attn_jvp_fwd_scored`` (constants; bounds and
    ``causal`` exclude each other: ``key_bounds`` combines masks); k, v, tk, tv may
    have fewer heads, of which q's are a multiple.  To capture forward and
    backward into a CUDA graph, give leaves that no live eager graph refers to
    (detached copies): autograd would run their accumulation on the eager stream."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    bounds = key_begin is not None or key_end is not None
    if bounds and causal:
        raise ValueError("causal goes into the bounds: key_bounds(Lq, Lk, causal=True, ...)")
    if softcap or slopes is not None or bounds or k.shape[1] != q.shape[1]:
        if causal:
            key_begin, key_end = key_bounds(q.shape[2], k.shape[2], causal=True, device=q.device)
        return AttnJvpScoredFunction.apply(q, k, v, tq, tk, tv, float(scale), float(softcap or 0.0), slopes, key_begin,
                                           key_end)
    return AttnJvpFunction.apply(q, k, v, tq, tk, tv, float(scale), bool(causal))
