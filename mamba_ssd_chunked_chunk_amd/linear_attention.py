"""Linear attention with a fixed decay per head as a differentiable torch
function, over the library's forward and backward passes (include/ssd.h,
ssd_linear_attn_varlen_fwd and _bwd)."""

from __future__ import annotations

import torch

from . import binding


def _aligned(g):
    """A gradient as the library takes it: dense, from a 16-byte boundary on (autograd may hand over part of a
    longer one)."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, query_start_loc, initial_states, scale, padded, state_dtype):
        new = torch.zeros if padded else torch.empty
        batch = query_start_loc.numel() - 1
        shape = (batch, v.shape[1], v.shape[2], q.shape[2])
        o = new(v.shape, dtype=v.dtype, device=v.device)
        final = torch.empty(shape, dtype=state_dtype if initial_states is None else initial_states.dtype,
                            device=v.device)
        binding.ssd_linear_attn_varlen_fwd(o, q, k, v, log_decay, initial_states, final, query_start_loc, scale=scale)
        ctx.save_for_backward(q, k, v, log_decay, query_start_loc, initial_states)
        ctx.scale, ctx.new, ctx.kind = scale, new, final.dtype
        ctx.set_materialize_grads(False)
        return o, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o, d_final):
        q, k, v, log_decay, query_start_loc, initial = ctx.saved_tensors
        if d_o is None and d_final is None:
            return (None,) * 9
        d_o = torch.zeros_like(v, memory_format=torch.contiguous_format) if d_o is None else _aligned(d_o)
        d_final = None if d_final is None else _aligned(d_final)
        dq, dk, dv = (ctx.new(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        batch = query_start_loc.numel() - 1
        d_initial = None
        if initial is not None and ctx.needs_input_grad[5]:
            d_initial = torch.empty((batch, v.shape[1], v.shape[2], q.shape[2]), dtype=ctx.kind, device=v.device)
        binding.ssd_linear_attn_varlen_bwd(dq, dk, dv, d_initial, q, k, v, d_o, log_decay, initial, d_final,
                                           query_start_loc, scale=ctx.scale)
        return dq, dk, dv, None, None, d_initial, None, None, None


def linear_attention(q, k, v, log_decay, query_start_loc, initial_states=None, *, scale=None, padded=False,
                     state_dtype=torch.float32):
    """o and final states of linear attention with decay exp(log_decay[h]) over a ragged batch:

        S_t = exp(log_decay[h]) S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t

    q, k bf16 [T,G,K], v bf16 [T,H,V] (slices of one projection will do), log_decay fp32 [H] (a constant of the
    layer: it gets no gradient), query_start_loc int32 [batch+1], initial_states [batch,H,V,K] in fp32 or bf16, or
    None for zero (the final states are then of ``state_dtype``; an empty tensor stands for zero too, in its own
    type).  ``scale``: None for K ** -0.5.  Returns o bf16 [T,H,V] and the final states [batch,H,V,K]; both are
    differentiable in q, k, v and initial_states.

    Rows behind query_start_loc[-1] need ``padded=True``: their outputs and gradients are then zero (otherwise they
    are not written).
    """
    if log_decay.requires_grad:
        raise ValueError("log_decay gets no gradient: pass it detached")
    if initial_states is not None and initial_states.numel() == 0:
        initial_states, state_dtype = None, initial_states.dtype
    return _LinearAttention.apply(q, k, v, log_decay, query_start_loc, initial_states,
                                  q.shape[-1] ** -0.5 if scale is None else scale, padded, state_dtype)
