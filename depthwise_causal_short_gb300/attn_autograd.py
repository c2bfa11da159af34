"""qk_norm_rope and decay_attention: the mixer's calls as differentiable PyTorch functions.

Only marshalling lives here, as in the convolution's causal_conv1d: the forward is one
cattn_*_fwd call, the backward one cattn_*_bwd call.  The gradients have no gradients of their own:
a second backward through them (create_graph=True) raises.
"""
from __future__ import annotations

import torch

from . import attn
from .autograd import once


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, positions, mode, eps, interleaved):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        ctx.kw = dict(mode=mode, eps=eps, interleaved=interleaved)
        return attn.cattn_qknorm_fwd(q, k, wq=wq, wk=wk, cos=cos, sin=sin, positions=positions,
                                     **ctx.kw)

    @staticmethod
    def backward(ctx, dyq, dyk):
        q, k, wq, wk, cos, sin, positions = ctx.saved_tensors
        dq, dk, dwq, dwk = attn.cattn_qknorm_bwd(q, k, dyq.contiguous(), dyk.contiguous(), wq=wq,
                                                 wk=wk, cos=cos, sin=sin, positions=positions,
                                                 **ctx.kw)
        need = ctx.needs_input_grad
        dq, dk, dwq, dwk = once("qk_norm_rope", (dq, dk, dwq, dwk), (dyq, dyk, q, k, wq, wk))
        return (dq if need[0] else None, dk if need[1] else None, dwq if need[2] else None,
                dwk if need[3] else None, None, None, None, None, None, None)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, wq: torch.Tensor | None = None,
                 wk: torch.Tensor | None = None, cos: torch.Tensor | None = None,
                 sin: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                 mode: str = "rms", eps: float = 1e-6, interleaved: bool = False):
    """Per-head norm of q [total, Hq, K] and k [total, Hk, K] with the position rotation, in one
    pass; differentiable in q, k and the weights.  See attn.cattn_qknorm_fwd."""
    return _QkNormRope.apply(q, k, wq, wk, cos, sin, positions, mode, eps, interleaved)


class _DecayAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, cu_seqlens, initial_state, scale, output_final_state):
        o, final, _ = attn.cattn_linear_fwd(q, k, v, g, cu_seqlens, scale=scale,
                                            initial_state=initial_state,
                                            final_state=bool(output_final_state))
        ctx.scale = scale
        ctx.save_for_backward(q, k, v, g, cu_seqlens, initial_state)
        if final is not None:
            ctx.mark_non_differentiable(final)
        return o, final

    @staticmethod
    def backward(ctx, do, _dfinal):
        q, k, v, g, cu_seqlens, initial_state = ctx.saved_tensors
        need = ctx.needs_input_grad
        want = initial_state is not None and need[5]
        dq, dk, dv, dg, ds = attn.cattn_linear_bwd(q, k, v, g, do.contiguous(), cu_seqlens,
                                                   scale=ctx.scale, initial_state=initial_state,
                                                   want_dinit=want)
        dq, dk, dv, dg, ds = once("decay_attention", (dq, dk, dv, dg, ds),
                                  (do, q, k, v, g, initial_state))
        return (dq if need[0] else None, dk if need[1] else None, dv if need[2] else None,
                dg if need[3] else None, None, ds if want else None, None, None)


def decay_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    cu_seqlens: torch.Tensor, initial_state: torch.Tensor | None = None,
                    scale: float | None = None, output_final_state: bool = False):
    """Linear attention with a decay for each token and head over packed sequences; returns (o,
    final_state or None).  Differentiable in q, k, v, g and initial_state [nseq, Hv, K, V]; the
    final state is a constant.  See attn.cattn_linear_fwd."""
    if initial_state is not None and initial_state.shape[0] != cu_seqlens.numel() - 1:
        raise ValueError("initial_state must hold one state per sequence")
    return _DecayAttention.apply(q, k, v, g, cu_seqlens, initial_state, scale, output_final_state)
