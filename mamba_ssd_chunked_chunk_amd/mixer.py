"""What a selective state space layer is made of, as differentiable torch
functions over the library's forward and backward passes (include/ssd.h):
``rms_norm`` with the residual's addition, ``causal_conv`` and
``selective_scan``.  A layer over a ragged batch is

    h, residual = rms_norm(x, weight, residual)
    u, z = in_proj(h).chunk(2, -1)
    u, conv_state = causal_conv(u, conv_weight, conv_bias, query_start_loc)
    dt, B, C = x_proj(u).split(...)
    y, state = selective_scan(u, dt_proj(dt), A, B, C, D, z, dt_bias, query_start_loc)

and x = out_proj(y) goes to the next one with the residual.  For serving, the
in-place forms of ``binding`` take the same tensors and the pools."""

from __future__ import annotations

import torch

from . import binding
from .linear_attention import _aligned


def _dense_input(t, step, align):
    """An input as the library takes it: a view with dense rows, whose stride is a multiple of ``step``, from a
    boundary of ``align`` bytes on; else a copy."""
    row, ok = 1, t.data_ptr() % align == 0
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        ok = ok and (n <= 1 or s == row)
        row *= n
    if ok and (t.shape[0] <= 1 or (t.stride(0) >= row and t.stride(0) % step == 0)):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        shape, width = x.shape, x.shape[-1]
        x = _dense_input(x.reshape(-1, width), 8, 16)
        weight = _aligned(weight)
        y = torch.empty((x.shape[0], width), dtype=torch.bfloat16, device=x.device)
        out = None
        if residual is not None:
            residual = _aligned(residual.reshape(-1, width))
            out = torch.empty_like(residual)
        binding.ssd_rms_norm_fwd(y, None, out, x, residual, weight, eps=eps)
        ctx.save_for_backward(x if out is None else out, weight)
        ctx.eps, ctx.shape, ctx.added = eps, shape, out is not None
        return (y.view(shape),) if out is None else (y.view(shape), out.view(shape))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_y, d_out=None):
        r, weight = ctx.saved_tensors
        if d_y is None and d_out is None:
            return (None,) * 4
        r = r.contiguous()
        dx = torch.empty(r.shape, dtype=torch.bfloat16, device=r.device)
        dw = torch.empty_like(weight)
        own = ctx.added and r.dtype == torch.float32 and ctx.needs_input_grad[2]
        d_residual = torch.empty_like(r) if own else None
        d_y = torch.zeros_like(dx) if d_y is None else _aligned(d_y.reshape(r.shape))
        d_out = None if d_out is None else _aligned(d_out.reshape(r.shape))
        binding.ssd_rms_norm_bwd(dx, d_residual, dw, r, weight, d_y, d_out, eps=ctx.eps)
        dx = dx.view(ctx.shape)
        if not ctx.added:
            return dx, dw, None, None
        return dx, dw, d_residual.view(ctx.shape) if own else dx if r.dtype == torch.bfloat16 else None, None


def rms_norm(x, weight, residual=None, *, eps=1e-5):
    """Root-mean-square norm of x bf16 [..., width], or of residual + x: returns y, or y and residual + x.

    ``residual`` (fp32 or bf16, the shape of x) is the residual stream, held in its own type: the sum is rounded to
    it once and y = r / sqrt(mean(r^2) + eps) * weight is the norm of what is stored.  weight fp32 [width].
    Differentiable in x, weight and residual.  (For an output in 8 bits: binding.ssd_rms_norm_fwd.)
    """
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual: expected shape {tuple(x.shape)}, got {tuple(residual.shape)}")
    r = _RmsNorm.apply(x, weight, residual, eps)
    return r[0] if residual is None else r


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, query_start_loc, initial_states, silu, padded):
        ctx.set_materialize_grads(False)
        new = torch.zeros if padded else torch.empty
        x, weight = _dense_input(x, 8, 16), _aligned(weight)
        bias = None if bias is None else _aligned(bias)
        initial_states = None if initial_states is None else _aligned(initial_states)
        y = new(x.shape, dtype=x.dtype, device=x.device)
        final = torch.empty((query_start_loc.numel() - 1, weight.shape[1] - 1, x.shape[1]), dtype=x.dtype,
                            device=x.device)
        binding.ssd_causal_conv_varlen_fwd(y, x, weight, bias, initial_states, final, query_start_loc, silu=silu)
        ctx.save_for_backward(x, weight, bias, query_start_loc, initial_states)
        ctx.silu, ctx.new = silu, new
        return y, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_y, d_final):
        x, weight, bias, query_start_loc, initial = ctx.saved_tensors
        if d_y is None and d_final is None:
            return (None,) * 7
        dx = ctx.new(x.shape, dtype=x.dtype, device=x.device)
        d_y = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if d_y is None else _aligned(d_y)
        d_final = None if d_final is None else _aligned(d_final)
        dw, db = torch.empty_like(weight), None if bias is None else torch.empty_like(bias)
        d_initial = torch.empty_like(initial) if initial is not None and ctx.needs_input_grad[4] else None
        binding.ssd_causal_conv_varlen_bwd(dx, dw, db, d_initial, x, weight, bias, d_y, initial, d_final,
                                           query_start_loc, silu=ctx.silu)
        return dx, dw, db, None, d_initial, None, None


def causal_conv(x, weight, bias, query_start_loc, initial_states=None, *, silu=True, padded=False):
    """Short causal depthwise convolution over a ragged batch, and the states it leaves:

        y_t = silu(bias + sum_j weight[:, j] x_{t - (width - 1) + j})

    x bf16 [T,channels] (a slice of a projection will do), weight fp32 [channels,width] with width 2 to 4, bias fp32
    [channels] or None, query_start_loc int32 [batch+1], initial_states bf16 [batch,width-1,channels] (the inputs
    ahead of each sequence, oldest first) or None (or empty) for zeros.  Returns y bf16 [T,channels] and the last
    inputs of each sequence [batch,width-1,channels]; differentiable in x, weight, bias and initial_states.

    Rows behind query_start_loc[-1] need ``padded=True``: their outputs and gradients are then zero (otherwise they
    are not written).
    """
    if initial_states is not None and initial_states.numel() == 0:
        initial_states = None
    return _CausalConv.apply(x, weight, bias, query_start_loc, initial_states, silu, padded)


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, query_start_loc, initial_states, dt_softplus, padded, state_dtype):
        ctx.set_materialize_grads(False)
        new = torch.zeros if padded else torch.empty
        x, dt = _dense_input(x, 8, 16), _dense_input(dt, 8, 16)
        z = None if z is None else _dense_input(z, 8, 16)
        B, C, A = _dense_input(B, 2, 4), _dense_input(C, 2, 4), _aligned(A)
        D, dt_bias = (None if t is None else t.contiguous() for t in (D, dt_bias))
        initial_states = None if initial_states is None else _aligned(initial_states)
        y = new(x.shape, dtype=x.dtype, device=x.device)
        final = torch.empty((query_start_loc.numel() - 1, *A.shape), device=x.device,
                            dtype=state_dtype if initial_states is None else initial_states.dtype)
        binding.ssd_selective_scan_varlen_fwd(y, x, dt, A, B, C, D, z, dt_bias, initial_states, final,
                                              query_start_loc, dt_softplus=dt_softplus)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, query_start_loc, initial_states)
        ctx.softplus, ctx.new, ctx.kind = dt_softplus, new, final.dtype
        return y, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_y, d_final):
        x, dt, A, B, C, D, z, dt_bias, query_start_loc, initial = ctx.saved_tensors
        if d_y is None and d_final is None:
            return (None,) * 13

        def rows(t):
            return None if t is None else ctx.new(t.shape, dtype=t.dtype, device=t.device)

        def vector(t):
            return None if t is None else torch.empty_like(t)

        d_y = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if d_y is None else _aligned(d_y)
        d_final = None if d_final is None else _aligned(d_final)
        dx, ddt, dB, dC, dz = rows(x), rows(dt), rows(B), rows(C), rows(z)
        dA, dD, d_bias = vector(A), vector(D), vector(dt_bias)
        d_initial = None
        if initial is not None and ctx.needs_input_grad[9]:
            d_initial = torch.empty(initial.shape, dtype=ctx.kind, device=x.device)
        binding.ssd_selective_scan_varlen_bwd(dx, ddt, dA, dB, dC, dD, dz, d_bias, d_initial, x, dt, A, B, C, D, z,
                                              dt_bias, d_y, initial, d_final, query_start_loc,
                                              dt_softplus=ctx.softplus)
        return dx, ddt, dA, dB, dC, dD, dz, d_bias, None, d_initial, None, None, None


def selective_scan(x, dt, A, B, C, D, z, dt_bias, query_start_loc, initial_states=None, *, dt_softplus=True,
                   padded=False, state_dtype=torch.float32):
    """Selective scan over a ragged batch, and the states it leaves.  For channel d of group g:

        h_t = exp(dts_t A) h_{t-1} + dts_t x_t B_t,   dts = softplus(dt + dt_bias)
        y_t = (C_t . h_t + D x_t) silu(z_t)

    x, dt, z bf16 [T,channels] (z None: no gate), B, C bf16 [T,G,N] (slices of projections will do), A fp32
    [channels,N], D and dt_bias fp32 [channels] or None, query_start_loc int32 [batch+1], initial_states
    [batch,channels,N] in fp32 or bf16, or None for zero (the final states are then of ``state_dtype``; an empty
    tensor stands for zero too, in its own type).  Returns y bf16 [T,channels] and the final states; differentiable in
    everything but query_start_loc.

    Rows behind query_start_loc[-1] need ``padded=True``: their outputs and gradients are then zero (otherwise they
    are not written).
    """
    if initial_states is not None and initial_states.numel() == 0:
        initial_states, state_dtype = None, initial_states.dtype
    return _SelectiveScan.apply(x, dt, A, B, C, D, z, dt_bias, query_start_loc, initial_states, dt_softplus, padded,
                                state_dtype)
