"""torch.autograd binding of the scan, the conv, the embedding and the residual block's operators.

The scan: forward through ssm_scan_fwd_save (the outputs plus the block checkpoints), backward through
ssm_scan_bwd_saved.

    from selective_state_space_76_amd import selective_scan
    out, last_state = selective_scan(u, delta, A, B, C, D, z, delta_bias)
    loss(out).backward()          # gradients of u, delta, A, B, C, D, z, delta_bias, initial_state

Bookkeeping only: the forward and backward arithmetic both run in the library's HIP kernels (the
gradients are the chain rule applied to the pages' forward recurrence, see include/ssm_scan.h).
Gradients are returned in each input's dtype; the library computes dA, dB, dC, dD and d(delta_bias)
in fp32 and they are cast to bf16 when those inputs are bf16.  Both discretisations (the default
dt*B and zero-order hold) and both scan directions have gradients.  There are no gradients of gradients: asking
for one (after create_graph=True) is an error.
"""
from __future__ import annotations

import functools

import torch

from ._lib import _io_dtype, checkpoints_shape, conv1d_fwd, scan_bwd, scan_fwd
from .block import (dropout_bwd, dropout_fwd, layer_norm_bwd, layer_norm_fwd, recurrence_bwd, recurrence_checkpoints_shape,
                    recurrence_fwd)
from .training import conv1d_bwd, embedding_bwd, embedding_fwd


class _NoSecond(torch.autograd.Function):
    """Passes n gradients on, as functions of the tensors behind them that cannot be differentiated."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tensors[:n]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of this package's operators cannot be differentiated again")


def _first_order(backward):
    """The kernels' results carry no graph.  Where the caller wants one (create_graph=True), the gradients are tied to
    everything that they depend on, so that a second derivative is refused and no term of it gets lost."""
    @functools.wraps(backward)
    def run(ctx, *douts):
        with torch.no_grad():
            grads = backward(ctx, *douts)
        if torch.is_grad_enabled():
            behind = [t for t in (*ctx.saved_tensors, *douts) if t is not None and t.requires_grad]
            some = [g for g in grads if g is not None]
            if behind and some:
                tied = iter(_NoSecond.apply(len(some), *some, *behind))
                grads = tuple(None if g is None else next(tied) for g in grads)
        return grads
    return run


def _dense(grad, dtype):
    """An output's gradient as the kernels take it: contiguous, from a multiple of 16 bytes on.  It may come as a view
    into a larger one, behind a concatenation for instance."""
    g = grad.to(dtype).contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class SelectiveScanFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, initial_state, zoh, reverse):
        # when a gradient will be asked for, the forward also writes the state entering every
        # 64-step block, and the backward starts from them instead of recomputing them
        ck = None
        if any(ctx.needs_input_grad[:9]):
            Bsz, Dm, L = u.shape
            ck = torch.empty(checkpoints_shape(Bsz, Dm, A.shape[1], L), dtype=torch.float32, device=u.device)
        out, final_state = scan_fwd(u, delta, A, B, C, D, z, delta_bias, initial_state, zoh=zoh, reverse=reverse,
                                    checkpoints=ck)
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, initial_state, ck)
        ctx.zoh, ctx.reverse = zoh, reverse
        return out, final_state

    @staticmethod
    @_first_order
    def backward(ctx, dout, dfinal):
        u, delta, A, B, C, D, z, delta_bias, initial_state, ck = ctx.saved_tensors
        dout = torch.zeros_like(u) if dout is None else _dense(dout, u.dtype)
        dfinal = None if dfinal is None else _dense(dfinal, torch.float32)
        g = scan_bwd(u, delta, A, B, C, D, z, delta_bias, initial_state, dout=dout, dfinal_state=dfinal,
                     zoh=ctx.zoh, reverse=ctx.reverse, checkpoints=ck)
        need = ctx.needs_input_grad

        def cast(grad, like, i):
            return grad.to(like.dtype) if (need[i] and grad is not None and like is not None) else None

        return (cast(g["du"], u, 0), cast(g["ddelta"], delta, 1), cast(g["dA"], A, 2), cast(g["dB"], B, 3),
                cast(g["dC"], C, 4), cast(g["dD"], D, 5), cast(g["dz"], z, 6), cast(g["ddelta_bias"], delta_bias, 7),
                cast(g["dinitial_state"], initial_state, 8), None, None)


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, initial_state=None, *, zoh=False,
                   reverse=False):
    """Differentiable selective scan.  Same arguments and layouts as scan_fwd; returns
    (out [B,D,L] in u's dtype, final_state [B,D,N] fp32)."""
    return SelectiveScanFn.apply(u, delta, A, B, C, D, z, delta_bias, initial_state, zoh, reverse)


class CausalConv1dFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state):
        u, final_state = conv1d_fwd(x, weight, bias, initial_state)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, initial_state)
        return u, final_state

    @staticmethod
    @_first_order
    def backward(ctx, dout, dfinal):
        x, weight, bias, initial_state = ctx.saved_tensors
        dout = torch.zeros_like(x) if dout is None else _dense(dout, x.dtype)
        dfinal = None if dfinal is None else _dense(dfinal, x.dtype)
        g = conv1d_bwd(x, weight, bias, initial_state, dout=dout, dfinal_state=dfinal)
        need = ctx.needs_input_grad
        # (an output without a gradient comes as None)
        return (g["dx"] if need[0] else None, g["dweight"] if need[1] else None,
                g["dbias"] if need[2] and bias is not None else None,
                g["dinitial_state"] if need[3] and initial_state is not None else None)


def causal_conv1d(x, weight, bias=None, initial_state=None):
    """Differentiable conv1d_fwd: (u [B,D,L], final_state [B,D,K-1]), with gradients of x, weight, bias and
    initial_state through conv1d_bwd."""
    return CausalConv1dFn.apply(x, weight, bias, initial_state)


class EmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, dtype, channels_first):
        ctx.save_for_backward(tokens)
        ctx.table = (weight.shape[0], weight.dtype, scale, channels_first)
        return embedding_fwd(tokens, weight, scale=scale, dtype=dtype, channels_first=channels_first)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        (tokens,) = ctx.saved_tensors
        rows, dtype, scale, channels_first = ctx.table
        dw = embedding_bwd(tokens, _dense(dout, dout.dtype), rows, scale=scale, channels_first=channels_first,
                           dtype=dtype)
        return None, dw, None, None, None


def embedding(tokens, weight, *, scale=1.0, dtype=None, channels_first=False):
    """Differentiable embedding_fwd; the gradient comes in weight's dtype, summed in fp32 and rounded once."""
    return EmbeddingFn.apply(tokens, weight, scale, dtype, channels_first)


def _seeds(seed):
    """(what is kept for the backward pass as a tensor, as a number)."""
    return (seed, None) if isinstance(seed, torch.Tensor) else (None, seed)


class LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, seed, eps, rms, channels_first, p, call):
        out, hidden, stats = layer_norm_fwd(x, weight, bias, residual, eps=eps, rms=rms, channels_first=channels_first, p=p,
                                            seed=seed, call=call)
        ctx.set_materialize_grads(False)
        ctx.x_dtype = x.dtype
        ctx.set = dict(rms=rms, channels_first=channels_first, p=p, call=call, residual=residual is not None,
                       bias=bias is not None)
        tensor, ctx.seed = _seeds(seed)
        ctx.save_for_backward(hidden, weight, stats, tensor)
        return (out,) if hidden is x else (out, hidden)

    @staticmethod
    @_first_order
    def backward(ctx, dout, dhidden=None):
        hidden, weight, stats, seed = ctx.saved_tensors
        seed = ctx.seed if seed is None else seed
        # (x's dtype is hidden's unless a residual in fp32 was added; an output without a gradient comes as None)
        dout = None if dout is None else _dense(dout, dout.dtype)
        dhidden = None if dhidden is None else _dense(dhidden, hidden.dtype)
        if dout is None:
            dout = torch.zeros(hidden.shape, dtype=ctx.x_dtype, device=hidden.device)
        g = layer_norm_bwd(dout, hidden, weight, stats, dhidden=dhidden, seed=seed, **ctx.set)
        need = ctx.needs_input_grad
        return (g["dx"] if need[0] else None, g["dweight"] if need[1] else None, g["dbias"] if need[2] else None,
                g["dresidual"] if need[3] else None, None, None, None, None, None, None)


def layer_norm(x, weight=None, bias=None, residual=None, *, eps=1e-5, rms=False, channels_first=False, p=0.0, seed=None,
               call=0):
    """Differentiable layer_norm_fwd.  Returns out, or (out, hidden) where there is a residual or dropout; hidden may go
    on as the residual of the next block, and its gradient is added on the way back."""
    got = LayerNormFn.apply(x, weight, bias, residual, seed, eps, rms, channels_first, p, call)
    return got if len(got) > 1 else got[0]


class DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, seed, p, call):
        tensor, ctx.seed = _seeds(seed)
        ctx.save_for_backward(tensor)
        ctx.set = (p, call, x.dtype)
        return dropout_fwd(x, p, seed, call=call, residual=residual)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        (seed,) = ctx.saved_tensors
        p, call, dtype = ctx.set
        dx = None
        if ctx.needs_input_grad[0]:
            dx = dropout_bwd(_dense(dout, dout.dtype), p, ctx.seed if seed is None else seed, call=call, dtype=dtype)
        return dx, dout if ctx.needs_input_grad[1] else None, None, None, None


def dropout(x, p, seed, *, call=0, residual=None):
    """Differentiable dropout_fwd: residual + dropout(x)."""
    return DropoutFn.apply(x, residual, seed, p, call)


class GatedRecurrenceFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, decay, r_bias, i_bias, z, initial_state, reverse):
        ck = None
        if any(ctx.needs_input_grad[:8]):
            ck = torch.empty(recurrence_checkpoints_shape(*x.shape, _io_dtype(x)), dtype=torch.float32, device=x.device)
        out, last = recurrence_fwd(x, r, i, decay, r_bias, i_bias, z, initial_state, reverse=reverse, checkpoints=ck)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, r, i, decay, r_bias, i_bias, z, initial_state, ck)
        ctx.reverse = reverse
        return out, last

    @staticmethod
    @_first_order
    def backward(ctx, dout, dlast):
        *ins, ck = ctx.saved_tensors
        dout = torch.zeros_like(ins[0]) if dout is None else _dense(dout, ins[0].dtype)
        dlast = None if dlast is None else _dense(dlast, torch.float32)
        g = recurrence_bwd(*ins, dout=dout, dfinal_state=dlast, reverse=ctx.reverse, checkpoints=ck)
        names = ("dx", "dr", "di", "ddecay", "dr_bias", "di_bias", "dz", "dinitial_state")
        return tuple(g[k] if need and t is not None else None
                     for k, t, need in zip(names, ins, ctx.needs_input_grad)) + (None,)


def gated_recurrence(x, r, i, decay, r_bias=None, i_bias=None, z=None, initial_state=None, *, reverse=False):
    """Differentiable recurrence_fwd: (out [B,D,L], final_state [B,D] fp32), with gradients of every tensor given."""
    return GatedRecurrenceFn.apply(x, r, i, decay, r_bias, i_bias, z, initial_state, reverse)
