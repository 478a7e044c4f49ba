"""The gated delta rule as a differentiable torch function (forward ``gdn_packed``, backward ``gdn_bwd``)."""
from __future__ import annotations

import torch

from . import binding


class _GatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, alpha, beta, S_in, cu_seqlens, status):
        o = S_out = None
        if cu_seqlens is not None and cu_seqlens.dim() == 1 and cu_seqlens.numel() and v.dim() == 3 and q.dim() == 3:
            # what no sequence covers is a value of the graph too, and not what the memory held
            o = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
            S_out = torch.zeros((cu_seqlens.numel() - 1, v.shape[1], v.shape[2], q.shape[2]), dtype=torch.float32, device=v.device)
        o, S_out = binding.gdn_packed(q, k, v, alpha, beta, cu_seqlens, S_in, o=o, S_out=S_out, return_state=True, status=status)
        ctx.save_for_backward(q, k, v, alpha, beta, S_in, cu_seqlens)
        ctx.status = status
        ctx.set_materialize_grads(False)
        return o, S_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, dS_out):
        q, k, v, alpha, beta, S_in, cu_seqlens = ctx.saved_tensors
        if do is None and dS_out is None:
            return (None,) * 8
        do = torch.zeros_like(v, memory_format=torch.contiguous_format) if do is None else do.contiguous()
        dS_out = None if dS_out is None else dS_out.contiguous()
        status = None if ctx.status is None else torch.empty_like(ctx.status)
        grads = binding.gdn_bwd(q, k, v, alpha, beta, do, cu_seqlens, S_in, dS_out=dS_out,
                                need_dS_in=S_in is not None and ctx.needs_input_grad[5], status=status)
        if status is not None:
            ctx.status |= status
        return tuple(g if need else None for g, need in zip(grads, ctx.needs_input_grad)) + (None, None)


def gated_delta_rule(q, k, v, alpha, beta, S_in=None, cu_seqlens=None, *, status=None):
    """o, S_out = the token-wise rule over B sequences of T tokens (q, k [B, T, Hk, d_k], v [B, T, H,
    d_v], alpha, beta [B, T, H]) or, with cu_seqlens (int32 [n + 1]), over n sequences packed into
    [N, heads, d] tensors; shapes, types and strides as in ``gdn_packed``.  S_in and S_out are fp32
    [sequences, H, d_v, d_k] (S_in None: zeros).  Differentiable in every floating input, once; the backward
    pass recomputes the forward.  o rows of tokens that no sequence covers are zeros, as are the S_out
    entries of sequences that are skipped (a range out of order or out of the tensors); ``status`` (a CUDA
    int32 tensor of one element) receives the GDN_SEQ_* bits of the forward pass, and the backward pass
    adds its own.
    """
    return _GatedDeltaRule.apply(q, k, v, alpha, beta, S_in, cu_seqlens, status)
