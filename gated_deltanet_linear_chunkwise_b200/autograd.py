"""The gated delta rule as a differentiable torch function (forward ``gdn_packed``, backward ``gdn_bwd``)."""
from __future__ import annotations

import torch

from . import binding


class _GatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, alpha, beta, S_in, cu_seqlens):
        o, S_out = binding.gdn_packed(q, k, v, alpha, beta, cu_seqlens, S_in, return_state=True)
        ctx.save_for_backward(q, k, v, alpha, beta, S_in, cu_seqlens)
        ctx.set_materialize_grads(False)
        return o, S_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, dS_out):
        q, k, v, alpha, beta, S_in, cu_seqlens = ctx.saved_tensors
        if do is None and dS_out is None:
            return (None,) * 7
        do = torch.zeros_like(v, memory_format=torch.contiguous_format) if do is None else do.contiguous()
        dS_out = None if dS_out is None else dS_out.contiguous()
        grads = binding.gdn_bwd(q, k, v, alpha, beta, do, cu_seqlens, S_in, dS_out=dS_out,
                                need_dS_in=S_in is not None and ctx.needs_input_grad[5])
        return tuple(g if need else None for g, need in zip(grads, ctx.needs_input_grad)) + (None,)


def gated_delta_rule(q, k, v, alpha, beta, S_in=None, cu_seqlens=None):
    """o, S_out = the token-wise rule over B sequences of T tokens (q, k [B, T, Hk, d_k], v [B, T, H,
    d_v], alpha, beta [B, T, H]) or, with cu_seqlens (int32 [n + 1]), over n sequences packed into
    [N, heads, d] tensors; shapes, types and strides as in ``gdn_packed``.  S_in and S_out are fp32
    [sequences, H, d_v, d_k] (S_in None: zeros).  Differentiable in every floating input, once; the backward
    pass recomputes the forward.  o rows of tokens that no sequence covers are not written.
    """
    return _GatedDeltaRule.apply(q, k, v, alpha, beta, S_in, cu_seqlens)
