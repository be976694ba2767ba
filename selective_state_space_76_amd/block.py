"""The operators of a residual block around the scan, the conv or the gated recurrence: the norm of the stream with a
branch added, dropout of that branch, and the recurrence itself.

    y, hidden, stats = layer_norm_fwd(branch, weight, bias, hidden, p=0.1, seed=s, call=k)   # hidden += dropout(branch)
    g = layer_norm_bwd(dy, hidden, weight, stats, dhidden=dh, residual=True, p=0.1, seed=s, call=k)
    out = dropout_fwd(branch, 0.1, s, call=k, residual=hidden)
    h, last = recurrence_fwd(x, r, i, decay, r_bias, i_bias, z)
    g = recurrence_bwd(x, r, i, decay, r_bias, i_bias, z, dout=dh)
    h_t = recurrence_update(last, x_t, r_t, i_t, decay, r_bias, i_bias, z_t)                 # one token

seed=: an int, or a tensor of one int64 on the device, which the kernels read: a graph that is to drop other elements at
every replay takes such a tensor and changes it.  With an int, which every replay would repeat, a forward call that drops
anything refuses to be captured.  call= tells the calls under one seed apart (a layer's number, say).

stream=: as in training.py.  This is argument marshalling: the arithmetic runs in the library's HIP kernels (see
include/ssm_scan.h for the formulas and layouts), and nothing falls back to anything else.
"""
from __future__ import annotations

import ctypes
from operator import index

import torch

from ._lib import (SSM_BF16, SSM_FLAG_REVERSE, _empty, _expect, _hand_out, _io_dtype, _launch, _nonempty, _ptr, _written,
                   load, ssm_dropout, ssm_norm_shape, ssm_recurrence_shape)
from .training import SSM_FLAG_CHANNELS_FIRST, _KIND, _address, _capturing, _queue, _stream, _workspace

SSM_FLAG_RMS = 4
_NONE = 0xFFFFFFFFFFFFFFFF


# Every tensor of a call is checked and turned into its address in one go.

def _arg(t, shape, dtype, name, device):
    """The address of a tensor that has to look like this (None for None); an error says what does not.  (Tensors that the
    call made itself are not looked at again.)"""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        _expect(t, shape, dtype, name, device)
        _ptr(t)
    return t.data_ptr()


def _like(t, dtype, stream):
    """An uninitialised tensor of t's shape; torch's quicker call where the dtype and the stream allow it.  (t is contiguous,
    or its call is refused.)"""
    if stream is None and dtype == t.dtype:
        return torch.empty_like(t)
    return _empty(t.shape, dtype, t.device, stream)


def _mask(p, seed, call, device, stream, fresh):
    """struct ssm_dropout, or None for no dropout.  fresh: a mask of this call, not that of an earlier one."""
    if p == 0.0:
        return None
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in [0, 1], got %r" % (p,))
    if seed is None:
        raise ValueError("dropout needs a seed")
    if type(seed) is not int and isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1:
            raise TypeError("seed: expected an int or one int64 on the device, got %s of %d" % (seed.dtype, seed.numel()))
        if seed.device != device:
            _expect(seed, seed.shape, seed.dtype, "seed", device)
        return ssm_dropout(p, 0, _ptr(seed), index(call) & _NONE)
    if fresh and _capturing(stream if device.index is None else _queue(stream, device.index)):
        raise RuntimeError("every replay would repeat this call's mask: give the seed as a tensor on the device")
    return ssm_dropout(p, index(seed) & _NONE, None, index(call) & _NONE)  # (numpy's integers, too)


def dropout_fwd(x, p, seed, *, call=0, residual=None, out=None, stream=None):
    """residual + dropout(x): each element of x (fp32 or bf16, any shape) is kept with probability 1 - p and then divided
    by it (p in steps of 1/65536).  residual: fp32 or bf16, x's shape.  Returns it in residual's dtype (without one: x's),
    rounded once."""
    device = x.device
    mask = _mask(p, seed, call, device, stream, True) or ssm_dropout()
    return _dropout(x, mask, residual, x.dtype if residual is None else residual.dtype, out, stream)


def dropout_bwd(dout, p, seed, *, call=0, dtype=None, dx=None, stream=None):
    """The gradient of dropout_fwd with respect to x, in `dtype` (default: dout's).  That of the residual is dout."""
    mask = _mask(p, seed, call, dout.device, stream, False) or ssm_dropout()
    return _dropout(dout, mask, None, dx.dtype if dx is not None and dtype is None else dtype or dout.dtype, dx, stream)


def _dropout(x, mask, residual, dtype, out, stream):
    n, device, made = x.numel(), x.device, None
    if n < 1:
        _nonempty(numel=n)
    kx, ko = _KIND.get(x.dtype), _KIND.get(dtype)
    if kx is None or ko is None:
        raise TypeError("streams must be float32 or bfloat16, got %s" % (x.dtype if kx is None else dtype))
    px, pr = _address(x), None if residual is None else _arg(residual, x.shape, dtype, "residual", device)
    if out is None:
        out = made = _like(x, dtype, stream)
        po = out.data_ptr()
    else:
        po = _arg(out, x.shape, dtype, "out", device)
    _launch(device, load().ssm_dropout_fwd, n, kx, ko, px, pr, mask, po, _stream(stream, device))
    if made is None:
        _written(out)
    if stream is not None:
        _hand_out(stream, made)
    return out


def _norm_shape(shape, x_dtype, hidden_dtype, rms, channels_first):
    """(struct ssm_norm_shape, rows, E)."""
    x, h = _KIND.get(x_dtype), _KIND.get(hidden_dtype)
    if x is None or h is None:
        raise TypeError("streams must be float32 or bfloat16, got %s" % (x_dtype if x is None else hidden_dtype))
    if x == 0 and h == 1:
        raise TypeError("residual and hidden: float32, or bfloat16 with x in bfloat16")
    flags = SSM_FLAG_RMS if rms else 0
    if channels_first:
        if len(shape) != 3:
            raise ValueError("channels_first: expected [B, E, L], got %d dimensions" % len(shape))
        B, E, L = shape
        if B < 1 or E < 1 or L < 1:
            _nonempty(batch=B, dim=E, seqlen=L)
        return ssm_norm_shape(B, L, E, x, h, flags | SSM_FLAG_CHANNELS_FIRST), B * L, E
    if len(shape) < 1:
        raise ValueError("expected [..., E], got no dimension")
    E, rows = shape[-1], 1
    for n in shape[:-1]:
        rows *= n
    if rows < 1 or E < 1:
        _nonempty(rows=rows, dim=E)
    return ssm_norm_shape(rows, 1, E, x, h, flags), rows, E


def layer_norm_fwd(x, weight=None, bias=None, residual=None, *, eps=1e-5, rms=False, channels_first=False, p=0.0,
                   seed=None, call=0, out=None, hidden=None, stats=None, stream=None):
    """(out, hidden, stats): hidden = residual + dropout(x), out = its layer norm, with rms=True its RMS norm.

    x: [..., E], with channels_first [B,E,L], fp32 or bf16; residual: the same shape, fp32 or x's dtype; weight, bias:
    [E] fp32, None for ones and zeros.  out comes in x's dtype, hidden in residual's (without a residual: x's; it is x
    itself where there is no dropout either), stats [2, rows] in fp32: the means (rms: zeros) and the factors
    1 / sqrt(variance + eps), for layer_norm_bwd; stats=False: not wanted.
    p, seed, call: dropout of x, as in dropout_fwd."""
    device, f32, shape, xdt = x.device, torch.float32, x.shape, x.dtype
    hdt = xdt if residual is None else residual.dtype
    sh, rows, E = _norm_shape(shape, xdt, hdt, rms, channels_first)
    mask = _mask(p, seed, call, device, stream, True) if p else None
    pr = _arg(residual, shape, hdt, "residual", device)
    pw, pb = _arg(weight, (E,), f32, "weight", device), _arg(bias, (E,), f32, "bias", device)
    plain = residual is None and mask is None
    if plain and hidden is not None:
        raise ValueError("hidden: without a residual and dropout it is x itself")
    px, given, made = _address(x), [], []
    if out is None:
        out = _like(x, xdt, stream)
        made.append(out)
        po = out.data_ptr()
    else:
        po = _arg(out, shape, xdt, "out", device)
        given.append(out)
    if plain:
        ph, hidden = None, x
    elif hidden is None:
        hidden = _like(x if residual is None else residual, hdt, stream)
        made.append(hidden)
        ph = hidden.data_ptr()
    else:
        ph = _arg(hidden, shape, hdt, "hidden", device)
        given.append(hidden)
    if stats is None:
        stats = _empty((2, rows), f32, device, stream)
        made.append(stats)
        pst = stats.data_ptr()
    else:
        stats = None if stats is False else stats
        pst = _arg(stats, (2, rows), f32, "stats", device)
        given.append(stats)
    _launch(device, load().ssm_layer_norm_fwd, sh, px, pw, pb, pr, eps, mask, po, ph, pst, _stream(stream, device))
    if given:
        _written(*given)
    if stream is not None:
        _hand_out(stream, *made)
    return out, hidden, stats


def layer_norm_bwd_workspace_size(dout, *, hidden_dtype=None, rms=False, channels_first=False) -> int:
    """Workspace bytes of layer_norm_bwd."""
    sh, _, _ = _norm_shape(dout.shape, dout.dtype, hidden_dtype or dout.dtype, rms, channels_first)
    return int(load().ssm_layer_norm_bwd_workspace_size(sh))


def layer_norm_bwd(dout, hidden, weight, stats, *, dhidden=None, rms=False, channels_first=False, p=0.0, seed=None, call=0,
                   residual=False, bias=True, x_dtype=None, grads=None, workspace=None, stream=None):
    """Gradients of layer_norm_fwd for the gradient dout of out and, optionally, dhidden of hidden (hidden's dtype), from
    what that call returned.  Returns a dict: dx (x_dtype, default dout's); dresidual (hidden's dtype; with residual=True);
    dweight (None without a weight) and dbias [E] in fp32 (bias=False: not computed).  Where nothing is dropped and the
    dtypes agree, dx is dresidual.  grads: optional dict of preallocated outputs with those names."""
    device, f32, shape, hdt = dout.device, torch.float32, dout.shape, hidden.dtype
    if x_dtype is not None and x_dtype != dout.dtype:
        raise TypeError("dout: expected x's dtype %s, got %s" % (x_dtype, dout.dtype))
    sh, rows, E = _norm_shape(shape, dout.dtype, hdt, rms, channels_first)
    mask = _mask(p, seed, call, device, stream, False) if p else None
    ph, pdh = _arg(hidden, shape, hdt, "hidden", device), _arg(dhidden, shape, hdt, "dhidden", device)
    pw, ps = _arg(weight, (E,), f32, "weight", device), _arg(stats, (2, rows), f32, "stats", device)
    one = residual and mask is None and hdt == dout.dtype
    g, made, to = dict(grads) if grads else {}, [], []
    for k, wanted, shp, dt in (("dx", not one, shape, dout.dtype), ("dresidual", residual, shape, hdt),
                               ("dweight", weight is not None, (E,), f32), ("dbias", bias, (E,), f32)):
        t = g.get(k)
        if not wanted:
            if t is not None and not (k == "dx" and t is g.get("dresidual")):
                raise ValueError("grads: %s is not computed here" % k)
            g[k] = None
            to.append(None)
        elif t is None:
            g[k] = t = _empty(shp, dt, device, stream) if k[1] in "wb" else _like(dout if k == "dx" else hidden, dt, stream)
            made.append(t)
            to.append(t.data_ptr())
        else:
            to.append(_arg(t, shp, dt, k, device))
    pd, lib, ws_bytes, pws = _address(dout), load(), 0, None
    if to[2] is not None or to[3] is not None:
        workspace, ws_bytes = _workspace(workspace, lib.ssm_layer_norm_bwd_workspace_size(sh), device, stream)
        pws = _address(workspace)
    _launch(device, lib.ssm_layer_norm_bwd, sh, pd, ph, pw, ps, pdh, mask, *to, pws, ws_bytes,
            _stream(stream, device))
    if grads:
        _written(*[g[k] for k in grads if k in ("dx", "dresidual", "dweight", "dbias")])
    if stream is not None:
        _hand_out(stream, *made)
    if one:
        g["dx"] = g["dresidual"]
    return g


def _recurrence_shape(x, reverse):
    if x.dim() != 3:
        raise ValueError("x: expected [B, D, L], got %d dimensions" % x.dim())
    B, D, L = x.shape
    if B < 1 or D < 1 or L < 1:
        _nonempty(batch=B, dim=D, seqlen=L)
    return ssm_recurrence_shape(B, D, L, _io_dtype(x), SSM_FLAG_REVERSE if reverse else 0), B, D


def _recurrence_args(x, r, i, decay, r_bias, i_bias, z, state, full, ends, device):
    """The addresses of a call's inputs, in the order of the C entry points."""
    dt, f32, D = x.dtype, torch.float32, (ends[1],)
    others = (_arg(r, full, dt, "r", device), _arg(i, full, dt, "i", device), _arg(decay, D, f32, "decay", device),
              _arg(r_bias, D, f32, "r_bias", device), _arg(i_bias, D, f32, "i_bias", device),
              _arg(z, full, dt, "z", device), _arg(state, ends, f32, "initial_state", device))
    return (_address(x), *others)


def recurrence_checkpoints_shape(batch, dim, seqlen, io_dtype=SSM_BF16):
    """Shape of the checkpoints that recurrence_fwd(checkpoints=...) writes and recurrence_bwd reads."""
    sh = ssm_recurrence_shape(batch, dim, seqlen, io_dtype, 0)
    return (batch, dim, int(load().ssm_recurrence_checkpoints(ctypes.byref(sh))))


def recurrence_workspace_size(batch, dim, seqlen, io_dtype=SSM_BF16) -> int:
    """Workspace bytes of recurrence_fwd."""
    return int(load().ssm_recurrence_workspace_size(ctypes.byref(ssm_recurrence_shape(batch, dim, seqlen, io_dtype, 0))))


def recurrence_bwd_workspace_size(batch, dim, seqlen, io_dtype=SSM_BF16, saved=False) -> int:
    """Workspace bytes of recurrence_bwd; saved=True: with the forward's checkpoints given."""
    sh = ssm_recurrence_shape(batch, dim, seqlen, io_dtype, 0)
    return int(load().ssm_recurrence_bwd_workspace_size(ctypes.byref(sh), 1 if saved else 0))


def recurrence_fwd(x, r, i, decay, r_bias=None, i_bias=None, z=None, initial_state=None, *, out=None, final_state=True,
                   reverse=False, checkpoints=None, workspace=None, stream=None):
    """The gated linear recurrence a = exp(-decay sigmoid(r + r_bias)), h = a h + sqrt(1 - a^2) sigmoid(i + i_bias) x,
    out = h silu(z).  x, r, i, z: [B,D,L] fp32 or bf16; decay (not negative), r_bias, i_bias: [D] fp32; initial_state:
    [B,D] fp32 or None.  Returns (out [B,D,L] in x's dtype, final_state [B,D] fp32 or None); final_state may be True
    (allocate), False/None (not written) or a tensor to write into.
    checkpoints: an fp32 tensor of recurrence_checkpoints_shape(...) to write for recurrence_bwd."""
    lib = load()
    sh, B, D = _recurrence_shape(x, reverse)
    device, given, made = x.device, (out, final_state, checkpoints), []
    ins = _recurrence_args(x, r, i, decay, r_bias, i_bias, z, initial_state, x.shape, (B, D), device)
    if out is None:
        out = _like(x, x.dtype, stream)
        made.append(out)
        po = out.data_ptr()
    else:
        po = _arg(out, x.shape, x.dtype, "out", device)
    if final_state is True:
        final_state = _empty((B, D), torch.float32, device, stream)
        made.append(final_state)
        pf = final_state.data_ptr()
    else:
        final_state = None if final_state is False else final_state
        pf = _arg(final_state, (B, D), torch.float32, "final_state", device)
    pc = None
    if checkpoints is not None:
        pc = _arg(checkpoints, (B, D, lib.ssm_recurrence_checkpoints(sh)), torch.float32, "checkpoints", device)
    need, ws_bytes, pws = lib.ssm_recurrence_workspace_size(sh), 0, None
    if need or workspace is not None:
        workspace, ws_bytes = _workspace(workspace, need, device, stream)
        pws = _address(workspace)
    _launch(device, lib.ssm_recurrence_fwd, sh, *ins, po, pf, pc, pws, ws_bytes, _stream(stream, device))
    _written(*given)
    if stream is not None:
        _hand_out(stream, *made)
    return out, final_state


def recurrence_bwd(x, r, i, decay, r_bias=None, i_bias=None, z=None, initial_state=None, *, dout, dfinal_state=None,
                   reverse=False, checkpoints=None, grads=None, workspace=None, stream=None):
    """Gradients of recurrence_fwd for the gradient dout [B,D,L] (x's dtype) of out and, optionally, dfinal_state [B,D]
    fp32.  Returns a dict: dx, dr, di, dz (x's dtype; dz None without z), ddecay, dr_bias, di_bias [D] (fp32, also without
    the biases: the gradients at zero) and dinitial_state [B,D] fp32.  grads: optional dict of preallocated outputs with
    those names.  checkpoints: what recurrence_fwd(checkpoints=...) wrote for the same inputs; without them the states
    are first made again."""
    lib = load()
    sh, B, D = _recurrence_shape(x, reverse)
    device, dt, f32, full = x.device, x.dtype, torch.float32, x.shape
    pd, pl = _arg(dout, full, dt, "dout", device), _arg(dfinal_state, (B, D), f32, "dfinal_state", device)
    pc = None
    if checkpoints is not None:
        pc = _arg(checkpoints, (B, D, lib.ssm_recurrence_checkpoints(sh)), f32, "checkpoints", device)
    ins = _recurrence_args(x, r, i, decay, r_bias, i_bias, z, initial_state, full, (B, D), device)
    g, made, to = dict(grads) if grads else {}, [], []
    outs = (("dx", full, dt), ("dr", full, dt), ("di", full, dt), ("dz", full, dt), ("ddecay", (D,), f32),
            ("dr_bias", (D,), f32), ("di_bias", (D,), f32), ("dinitial_state", (B, D), f32))
    for k, shp, d in outs:
        t = g.get(k)
        if k == "dz" and z is None:
            g[k] = None
            to.append(None)
        elif t is None:
            g[k] = t = _like(x, dt, stream) if shp is full else _empty(shp, d, device, stream)
            made.append(t)
            to.append(t.data_ptr())
        else:
            to.append(_arg(t, shp, d, k, device))
    need = lib.ssm_recurrence_bwd_workspace_size(sh, 0 if pc is None else 1)
    workspace, ws_bytes = _workspace(workspace, need, device, stream)
    _launch(device, lib.ssm_recurrence_bwd, sh, *ins, pd, pl, pc, *to, _address(workspace), ws_bytes,
            _stream(stream, device))
    if grads:
        _written(*[g[k] for k, _, _ in outs if k in grads])
    if stream is not None:
        _hand_out(stream, *made)
    return g


def recurrence_update(state, x, r, i, decay, r_bias=None, i_bias=None, z=None, *, out=None, stream=None):
    """One generation step of the recurrence: state [B,D] fp32 is updated in place; x, r, i, z: [B,D].  Returns out [B,D]
    in x's dtype."""
    if x.dim() != 2:
        raise ValueError("x: expected [B, D], got %d dimensions" % x.dim())
    B, D = size = x.shape
    if B < 1 or D < 1:
        _nonempty(batch=B, dim=D)
    device, dt, f32, made = x.device, x.dtype, torch.float32, None
    io = _KIND.get(dt)
    if io is None:
        _io_dtype(x)
    ps = _arg(state, size, f32, "state", device)
    ins = (_arg(r, size, dt, "r", device), _arg(i, size, dt, "i", device), _arg(decay, (D,), f32, "decay", device),
           _arg(r_bias, (D,), f32, "r_bias", device), _arg(i_bias, (D,), f32, "i_bias", device),
           _arg(z, size, dt, "z", device))
    px = _address(x)
    if out is None:
        out = made = _like(x, dt, stream)
        po = out.data_ptr()
    else:
        po = _arg(out, size, dt, "out", device)
    _launch(device, load().ssm_recurrence_update, B, D, io, ps, px, *ins, po, _stream(stream, device))
    torch._C._increment_version((state,) if made is not None else (state, out))  # (_written() in its cheapest form)
    if stream is not None:
        _hand_out(stream, made)
    return out
