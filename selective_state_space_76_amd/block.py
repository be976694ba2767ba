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

import torch

from ._lib import (SSM_BF16, SSM_FLAG_REVERSE, _check, _empty, _expect, _hand_out, _io_dtype, _nonempty, _ptr, load,
                   ssm_dropout, ssm_norm_shape, ssm_recurrence_shape)
from .training import (SSM_FLAG_CHANNELS_FIRST, _KIND, _address, _capturing, _stream, _want, _workspace)

SSM_FLAG_RMS = 4
_NONE = 0xFFFFFFFFFFFFFFFF


def _mask(p, seed, call, device, stream, fresh):
    """struct ssm_dropout, or None for no dropout.  fresh: a mask of this call, not that of an earlier one."""
    if p == 0.0:
        return None
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in [0, 1], got %r" % (p,))
    if seed is None:
        raise ValueError("dropout needs a seed")
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1:
            raise TypeError("seed: expected an int or one int64 on the device, got %s of %d" % (seed.dtype, seed.numel()))
        if seed.device != device:
            _expect(seed, seed.shape, seed.dtype, "seed", device)
        return ssm_dropout(p, 0, _ptr(seed), call & _NONE)
    if fresh and _capturing(stream):
        raise RuntimeError("every replay would repeat this call's mask: give the seed as a tensor on the device")
    return ssm_dropout(p, seed & _NONE, None, call & _NONE)


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


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
    kinds = _KIND.get(x.dtype), _KIND.get(dtype)
    if None in kinds:
        raise TypeError("streams must be float32 or bfloat16, got %s" % (x.dtype if kinds[0] is None else dtype))
    _want(residual, x.shape, dtype, "residual", device)
    if out is None:
        out = made = _empty(x.shape, dtype, device, stream)
    else:
        _want(out, x.shape, dtype, "out", device)
    _check(load().ssm_dropout_fwd(n, *kinds, _address(x), _address(residual), ctypes.byref(mask), _address(out),
                                  _stream(stream, device)))
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
    device, f32, shape = x.device, torch.float32, x.shape
    hdt = x.dtype if residual is None else residual.dtype
    sh, rows, E = _norm_shape(shape, x.dtype, hdt, rms, channels_first)
    mask = _mask(p, seed, call, device, stream, True)
    _want(residual, shape, hdt, "residual", device)
    _want(weight, (E,), f32, "weight", device)
    _want(bias, (E,), f32, "bias", device)
    made = []
    if out is None:
        out = _empty(shape, x.dtype, device, stream)
        made.append(out)
    else:
        _want(out, shape, x.dtype, "out", device)
    if residual is None and mask is None:
        if hidden is not None:
            raise ValueError("hidden: without a residual and dropout it is x itself")
        kept, hidden = None, x
    elif hidden is None:
        kept = hidden = _empty(shape, hdt, device, stream)
        made.append(hidden)
    else:
        _want(hidden, shape, hdt, "hidden", device)
        kept = hidden
    if stats is None:
        stats = _empty((2, rows), f32, device, stream)
        made.append(stats)
    elif stats is False:
        stats = None
    else:
        _want(stats, (2, rows), f32, "stats", device)
    _check(load().ssm_layer_norm_fwd(ctypes.byref(sh), _address(x), _address(weight), _address(bias), _address(residual),
                                     eps, _ref(mask), _address(out), _address(kept), _address(stats),
                                     _stream(stream, device)))
    _hand_out(stream, *made)
    return out, hidden, stats


def layer_norm_bwd_workspace_size(dout, *, hidden_dtype=None, channels_first=False) -> int:
    """Workspace bytes of layer_norm_bwd."""
    sh, _, _ = _norm_shape(dout.shape, dout.dtype, hidden_dtype or dout.dtype, False, channels_first)
    return int(load().ssm_layer_norm_bwd_workspace_size(ctypes.byref(sh)))


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
    mask = _mask(p, seed, call, device, stream, False)
    _want(hidden, shape, hdt, "hidden", device)
    _want(dhidden, shape, hdt, "dhidden", device)
    _want(weight, (E,), f32, "weight", device)
    _want(stats, (2, rows), f32, "stats", device)
    one = residual and mask is None and hdt == dout.dtype
    g, made = dict(grads) if grads else {}, []
    for k, wanted, shp, dt in (("dx", not one, shape, dout.dtype), ("dresidual", residual, shape, hdt),
                               ("dweight", weight is not None, (E,), f32), ("dbias", bias, (E,), f32)):
        if not wanted:
            if g.get(k) is not None and not (k == "dx" and g[k] is g.get("dresidual")):
                raise ValueError("grads: %s is not computed here" % k)
            g[k] = None
        elif g.get(k) is None:
            g[k] = _empty(shp, dt, device, stream)
            made.append(g[k])
        else:
            _want(g[k], shp, dt, k, device)
    lib, ws_bytes = load(), 0
    if g["dweight"] is not None or g["dbias"] is not None:
        workspace, ws_bytes = _workspace(workspace, lib.ssm_layer_norm_bwd_workspace_size(ctypes.byref(sh)), device, stream)
    _check(lib.ssm_layer_norm_bwd(ctypes.byref(sh), _address(dout), _address(hidden), _address(weight), _address(stats),
                                  _address(dhidden), _ref(mask), _address(g["dx"]), _address(g["dresidual"]),
                                  _address(g["dweight"]), _address(g["dbias"]), _address(workspace), ws_bytes,
                                  _stream(stream, device)))
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
    device, dt, f32, full, made = x.device, x.dtype, torch.float32, x.shape, []
    for t, shp, d, name in ((r, full, dt, "r"), (i, full, dt, "i"), (z, full, dt, "z"), (decay, (D,), f32, "decay"),
                            (r_bias, (D,), f32, "r_bias"), (i_bias, (D,), f32, "i_bias"),
                            (initial_state, (B, D), f32, "initial_state")):
        _want(t, shp, d, name, device)
    if out is None:
        out = _empty(full, dt, device, stream)
        made.append(out)
    else:
        _want(out, full, dt, "out", device)
    if final_state is True:
        final_state = _empty((B, D), f32, device, stream)
        made.append(final_state)
    elif final_state is False:
        final_state = None
    else:
        _want(final_state, (B, D), f32, "final_state", device)
    if checkpoints is not None:
        _want(checkpoints, (B, D, lib.ssm_recurrence_checkpoints(ctypes.byref(sh))), f32, "checkpoints", device)
    need, ws_bytes = lib.ssm_recurrence_workspace_size(ctypes.byref(sh)), 0
    if need or workspace is not None:
        workspace, ws_bytes = _workspace(workspace, need, device, stream)
    _check(lib.ssm_recurrence_fwd(ctypes.byref(sh), _address(x), _address(r), _address(i), _address(decay),
                                  _address(r_bias), _address(i_bias), _address(z), _address(initial_state), _address(out),
                                  _address(final_state), _address(checkpoints), _address(workspace), ws_bytes,
                                  _stream(stream, device)))
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
    for t, shp, d, name in ((r, full, dt, "r"), (i, full, dt, "i"), (z, full, dt, "z"), (decay, (D,), f32, "decay"),
                            (r_bias, (D,), f32, "r_bias"), (i_bias, (D,), f32, "i_bias"),
                            (initial_state, (B, D), f32, "initial_state"), (dout, full, dt, "dout"),
                            (dfinal_state, (B, D), f32, "dfinal_state")):
        _want(t, shp, d, name, device)
    if checkpoints is not None:
        _want(checkpoints, (B, D, lib.ssm_recurrence_checkpoints(ctypes.byref(sh))), f32, "checkpoints", device)
    g, made = dict(grads) if grads else {}, []
    for k, shp, d in (("dx", full, dt), ("dr", full, dt), ("di", full, dt), ("dz", full, dt), ("ddecay", (D,), f32),
                      ("dr_bias", (D,), f32), ("di_bias", (D,), f32), ("dinitial_state", (B, D), f32)):
        if k == "dz" and z is None:
            g[k] = None
        elif g.get(k) is None:
            g[k] = _empty(shp, d, device, stream)
            made.append(g[k])
        else:
            _want(g[k], shp, d, k, device)
    need = lib.ssm_recurrence_bwd_workspace_size(ctypes.byref(sh), 0 if checkpoints is None else 1)
    workspace, ws_bytes = _workspace(workspace, need, device, stream)
    _check(lib.ssm_recurrence_bwd(ctypes.byref(sh), _address(x), _address(r), _address(i), _address(decay),
                                  _address(r_bias), _address(i_bias), _address(z), _address(initial_state), _address(dout),
                                  _address(dfinal_state), _address(checkpoints), _address(g["dx"]), _address(g["dr"]),
                                  _address(g["di"]), _address(g["dz"]), _address(g["ddecay"]), _address(g["dr_bias"]),
                                  _address(g["di_bias"]), _address(g["dinitial_state"]), _address(workspace), ws_bytes,
                                  _stream(stream, device)))
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
    io, device, dt, f32, made = _io_dtype(x), x.device, x.dtype, torch.float32, None
    for t, shp, d, name in ((state, size, f32, "state"), (r, size, dt, "r"), (i, size, dt, "i"), (z, size, dt, "z"),
                            (decay, (D,), f32, "decay"), (r_bias, (D,), f32, "r_bias"), (i_bias, (D,), f32, "i_bias")):
        _want(t, shp, d, name, device)
    if out is None:
        out = made = _empty(size, dt, device, stream)
    else:
        _want(out, size, dt, "out", device)
    _check(load().ssm_recurrence_update(B, D, io, _address(state), _address(x), _address(r), _address(i), _address(decay),
                                        _address(r_bias), _address(i_bias), _address(z), _address(out),
                                        _stream(stream, device)))
    _hand_out(stream, made)
    return out
