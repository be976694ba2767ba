"""The training operators next to the scan: the conv's gradients, the embedding with its gradient, AdamW.

    x = embedding_fwd(tokens, table, scale=s, channels_first=True)       # [B,E,L], what the conv reads
    g = conv1d_bwd(x, weight, bias, dout=du)                             # dx, dweight, dbias, dinitial_state
    dtable = embedding_bwd(tokens, g["dx"], table.shape[0], scale=s, channels_first=True)
    opt = AdamW(params, lr=1e-4, weight_decay=0.1, state_bits=8, max_grad_norm=1.0)
    opt.step()

stream=: the kernels' stream, by default the current one.  To order it with the work that made the inputs (an AdamW
included) and with what uses the outputs is the caller's part, as with every stream.

As in _lib.py this is argument marshalling: the arithmetic runs in the library's HIP kernels (see
include/ssm_scan.h for the formulas and layouts), and nothing falls back to anything else.
"""
from __future__ import annotations

import ctypes
import math
import operator

import numpy as np
import torch
from torch.autograd.graph import increment_version

from ._lib import (SSM_BF16, SSM_F32, SSMError, _check, _empty, _expect, _hand_out, _io_dtype, _nonempty, _ptr, load,
                   ssm_adamw_config, ssm_embed_shape)

SSM_I32 = 0
SSM_I64 = 1
SSM_FLAG_CHANNELS_FIRST = 1
SSM_FLAG_ACCUMULATE = 2
ADAMW_BLOCK = 128
_KIND = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}
_dtype = operator.attrgetter("dtype")
_INDEX = {torch.int32: SSM_I32, torch.int64: SSM_I64}


# Small calls are bound by the host, so the checks of _lib.py are made in their cheapest order here: plain numbers
# for addresses, and _expect() (which says what is wrong) only where something is.

def _address(t):
    """The tensor's address, None for None; _ptr() refuses what is not on the GPU or not contiguous."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        _ptr(t)
    return t.data_ptr()


def _aligned(t, name):
    if t.data_ptr() % 16:
        raise SSMError(4, "%s does not begin at a multiple of 16 bytes" % name)


def _want(t, shape, dtype, name, device):
    if t is not None and (t.shape != shape or t.dtype != dtype or t.device != device):
        _expect(t, shape, dtype, name, device)


def _stream(stream, device):
    """The caller's stream, by default the current one of the tensors' device, as the number the library takes."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _capturing(stream):
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _workspace(workspace, need, device, stream):
    """The caller's workspace, or one made here."""
    if workspace is None:
        workspace = _empty(max(need, 1), torch.uint8, device, stream)
    elif workspace.device != device:
        raise ValueError("workspace: expected a tensor on %s, got %s" % (device, workspace.device))
    return workspace, workspace.numel() * workspace.element_size()


def conv1d_bwd_workspace_size(batch, dim, seqlen, width, io_dtype=SSM_BF16) -> int:
    """Workspace bytes of conv1d_bwd."""
    return int(load().ssm_conv1d_bwd_workspace_size(batch, dim, seqlen, width, io_dtype))


def conv1d_bwd(x, weight, bias=None, initial_state=None, *, dout, dfinal_state=None, grads=None, workspace=None,
               stream=None):
    """Gradients of conv1d_fwd for the gradient dout [B,D,L] of u and, optionally, dfinal_state [B,D,K-1] of
    the final state (both in x's dtype).  Returns a dict: dx [B,D,L] and dinitial_state [B,D,K-1] in
    x's dtype, dweight [D,K] and dbias [D] in fp32 (dbias also without a bias: the gradient at zero).
    grads: optional dict of preallocated outputs with those names."""
    lib = load()
    Bsz, Dm, L = x.shape
    K = weight.shape[1]
    if Bsz < 1 or Dm < 1 or L < 1 or K < 1:
        _nonempty(batch=Bsz, dim=Dm, seqlen=L, width=K)
    io, device, xdt, f32 = _io_dtype(x), x.device, x.dtype, torch.float32
    full, state, taps, channels = (Bsz, Dm, L), (Bsz, Dm, K - 1), (Dm, K), (Dm,)
    _want(weight, taps, f32, "weight", device)
    _want(bias, channels, f32, "bias", device)
    _want(initial_state, state, xdt, "initial_state", device)
    _want(dout, full, xdt, "dout", device)
    _want(dfinal_state, state, xdt, "dfinal_state", device)
    g, made = dict(grads) if grads else {}, []
    for k, shp, dt in (("dx", full, xdt), ("dweight", taps, f32), ("dbias", channels, f32),
                       ("dinitial_state", state, xdt)):
        if g.get(k) is None:
            g[k] = _empty(shp, dt, device, stream)
            made.append(g[k])
        else:
            _want(g[k], shp, dt, k, device)
    workspace, ws_bytes = _workspace(workspace, lib.ssm_conv1d_bwd_workspace_size(Bsz, Dm, L, K, io), device, stream)
    _check(lib.ssm_conv1d_bwd(Bsz, Dm, L, K, io, _address(x), _address(weight), _address(bias),
                              _address(initial_state), _address(dout), _address(dfinal_state), _address(g["dx"]),
                              _address(g["dweight"]), _address(g["dbias"]), _address(g["dinitial_state"]),
                              _address(workspace), ws_bytes, _stream(stream, device)))
    _hand_out(stream, *made)
    return g


def _embed_shape(tokens, rows, dim, table_dtype, io_dtype, channels_first, accumulate=False, scale=1.0):
    index, table, io = _INDEX.get(tokens.dtype), _KIND.get(table_dtype), _KIND.get(io_dtype)
    if index is None:
        raise TypeError("tokens must be int32 or int64, got %s" % tokens.dtype)
    if table is None or io is None:
        raise TypeError("tables and embeddings must be float32 or bfloat16, got %s"
                        % (table_dtype if table is None else io_dtype))
    size = tokens.shape
    if len(size) not in (1, 2):
        raise ValueError("tokens: expected [B, L] or [T], got %d dimensions" % len(size))
    if channels_first and len(size) != 2:
        raise ValueError("channels_first needs tokens of shape [B, L]")
    Bsz, L = size if len(size) == 2 else (1, size[0])
    if Bsz < 1 or L < 1 or rows < 1 or dim < 1:
        _nonempty(batch=Bsz, seqlen=L, rows=rows, dim=dim)
    if not math.isfinite(scale):
        raise ValueError("scale must be finite, got %r" % (scale,))
    flags = (SSM_FLAG_CHANNELS_FIRST if channels_first else 0) | (SSM_FLAG_ACCUMULATE if accumulate else 0)
    return (ssm_embed_shape(Bsz, L, rows, dim, index, table, io, flags),
            (Bsz, dim, L) if channels_first else (*size, dim))


def embedding_fwd(tokens, weight, *, scale=1.0, dtype=None, channels_first=False, out=None, stream=None):
    """scale * weight[tokens].  tokens: int32 or int64, [B,L], or [T] (the single tokens of a generation step);
    weight: [V,E] fp32 or bf16; a token outside [0, V) gives zeros.  Returns [B,L,E] (or [T,E]), with channels_first
    [B,E,L], in `dtype` (default: weight's), rounded once."""
    lib = load()
    dtype = out.dtype if out is not None and dtype is None else dtype or weight.dtype
    if weight.dim() != 2:
        raise ValueError("weight: expected [V, E], got %d dimensions" % weight.dim())
    rows, dim = weight.shape
    sh, shape = _embed_shape(tokens, rows, dim, weight.dtype, dtype, channels_first, scale=scale)
    device, made = tokens.device, None
    if out is None:
        out = made = _empty(shape, dtype, device, stream)
    else:
        _want(out, shape, dtype, "out", device)
    if weight.device != device:
        _expect(weight, weight.shape, weight.dtype, "weight", device)
    _check(lib.ssm_embedding_fwd(ctypes.byref(sh), _address(tokens), _address(weight), scale, _address(out),
                                 _stream(stream, device)))
    _hand_out(stream, made)
    return out


def embedding_bwd_workspace_size(tokens, dout, rows, *, dtype=torch.float32, channels_first=False) -> int:
    """Workspace bytes of embedding_bwd for these arguments."""
    dim = dout.shape[1 if channels_first else -1]
    sh, _ = _embed_shape(tokens, rows, dim, dtype, dout.dtype, channels_first)
    return int(load().ssm_embedding_bwd_workspace_size(ctypes.byref(sh)))


def embedding_bwd(tokens, dout, rows, *, scale=1.0, channels_first=False, dtype=None, dweight=None, accumulate=False,
                  workspace=None, stream=None):
    """Gradient of embedding_fwd with respect to a table of `rows` rows: for every token, scale times the sum of its
    positions' rows of dout ([B,L,E], [T,E] or with channels_first [B,E,L]; fp32 or bf16), summed in fp32 in a fixed
    order.  Returns dweight [rows,E] in `dtype` (default fp32); accumulate=True adds to the dweight given, of which
    only the rows of tokens that occur are touched."""
    lib = load()
    if accumulate and dweight is None:
        raise ValueError("accumulate needs the dweight to add to")
    dtype = dweight.dtype if dweight is not None and dtype is None else dtype or torch.float32
    want = 3 if channels_first else tokens.dim() + 1
    if dout.dim() != want:
        raise ValueError("dout: expected %d dimensions, got %d" % (want, dout.dim()))
    dim = dout.shape[1 if channels_first else -1]
    sh, shape = _embed_shape(tokens, rows, dim, dtype, dout.dtype, channels_first, accumulate, scale)
    device, made = tokens.device, None
    _want(dout, shape, dout.dtype, "dout", device)
    if dweight is None:
        dweight = made = _empty((rows, dim), dtype, device, stream)
    _want(dweight, (rows, dim), dtype, "dweight", device)
    need = int(lib.ssm_embedding_bwd_workspace_size(ctypes.byref(sh)))
    workspace, ws_bytes = _workspace(workspace, need, device, stream)
    _check(lib.ssm_embedding_bwd(ctypes.byref(sh), _address(tokens), _address(dout), scale, _address(dweight),
                                 _address(workspace), ws_bytes, _stream(stream, device)))
    _hand_out(stream, made)
    return dweight


# struct ssm_adamw_tensor
_TENSOR = np.dtype([("param", "u8"), ("grad", "u8"), ("numel", "i8"), ("offset", "i8"), ("param_dtype", "i4"),
                    ("grad_dtype", "i4")])


class AdamW:
    """AdamW over many tensors at once, in place, with decoupled weight decay and bias-corrected moments.

    params: fp32 or bf16 tensors on one GPU, contiguous, from multiples of 16 bytes on (and so the gradients).  lr, betas,
    eps, weight_decay and max_grad_norm are attributes that may be changed between steps.
    state_bits: 32 (fp32 moments) or 8 (one byte per element and an int16 per 128; see include/ssm_scan.h).
    master_weights: fp32 copies of the bf16 parameters, on which the step works; without them a bf16 parameter is
        rounded stochastically (to nearest, updates under half a unit would be lost).
    max_grad_norm: scale the gradients so that their norm over all tensors is at most this; a step whose
        norm is not finite changes nothing and is not counted.
    seed: of the stochastic rounding (a hash of seed, step, tensor and element: the same on every run).
    A step may be captured in a graph where max_grad_norm is set (math.inf where nothing is to be clipped): every replay
    is then the next step, with the addresses, lr and other settings of the capture.  Without it the number of the
    step is an argument of the kernels, which every replay would repeat, and a capture is refused.
    state, step: state_dict()'s tensors to go on from (taken over, not copied), and the steps already made.

    The states of all tensors are flat buffers: tensor k's begin at offsets[k], a multiple of 128."""

    def __init__(self, params, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32,
                 master_weights=True, max_grad_norm=None, seed=0, state=None, step=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits, self.max_grad_norm = state_bits, max_grad_norm
        self.seed = int(seed)
        self.device = self.params[0].device
        for p in self.params:
            _io_dtype(p)
            _ptr(p)
            _aligned(p, "a parameter")
            if p.numel() < 1:
                raise ValueError("empty parameter")
            if p.device != self.device:
                raise ValueError("parameters on %s and %s" % (self.device, p.device))
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size()) for p in self.params)
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("parameters overlap")
        self._shapes = [p.shape for p in self.params]
        self._dtypes = [p.dtype for p in self.params]
        self._grad_dtypes = None  # those that the table says
        n = np.array([p.numel() for p in self.params], np.int64)
        room = -(-n // ADAMW_BLOCK) * ADAMW_BLOCK
        self.offsets = (np.cumsum(room) - room).tolist()
        self.numel = int(room.sum())
        self._table = np.zeros(len(n), _TENSOR)
        self._table["numel"], self._table["offset"] = n, self.offsets
        self._table["param_dtype"] = [_io_dtype(p) for p in self.params]
        want = {"exp_avg": (self.numel, torch.float32 if state_bits == 32 else torch.uint8)}
        want["exp_avg_sq"] = want["exp_avg"]
        if state_bits == 8:
            want["exp_avg_base"] = want["exp_avg_sq_base"] = (self.numel // ADAMW_BLOCK, torch.int16)
        if master_weights and torch.bfloat16 in self._dtypes:
            want["master"] = (self.numel, torch.float32)
        given = {k: v for k, v in (state or {}).items() if v is not None}
        if set(given) - set(want):
            raise ValueError("state: %s not expected here" % ", ".join(sorted(set(given) - set(want))))
        self.state = {}
        # With max_grad_norm the device counts the steps, which of them it leaves out is known only there; else _count.
        self._progress = torch.zeros(4, dtype=torch.int64, device=self.device)  # struct ssm_adamw_progress
        self._count = int(step)
        if max_grad_norm is not None:
            self._count_on_device(None)
        for k, (size, dt) in want.items():
            t = given.get(k)
            if t is None:
                t = torch.zeros(size, dtype=dt, device=self.device)
                if k == "master":
                    for p, o in zip(self.params, self.offsets):
                        t[o:o + p.numel()].copy_(p.detach().reshape(-1))
            _expect(t, (size,), dt, k, self.device)
            _ptr(t)
            _aligned(t, k)
            self.state[k] = t

    @property
    def step_count(self):
        """The number of steps made.  With max_grad_norm this waits for the GPU."""
        if self._count is not None:
            return self._count
        torch.cuda.synchronize(self.device)
        return int(self._progress[0])

    def _count_on_device(self, stream):
        with torch.cuda.stream(stream):
            self._progress[:1].fill_(self._count)
        self._count = None

    def state_dict(self):
        """The state tensors and the number of steps made: AdamW(params, **settings, **state_dict) goes on from here."""
        return {"state": dict(self.state), "step": self.step_count}

    def _checked(self, tensors, what):
        """Their addresses; every call looks at shape, device and layout anew (and the caller at the types)."""
        if list(map(torch.Tensor.size, tensors)) != self._shapes:
            raise ValueError("%s: shapes differ from the parameters' at construction" % what)
        if set(map(torch.Tensor.get_device, tensors)) != {self.device.index}:
            raise ValueError("%s: expected tensors on %s" % (what, self.device))
        if not all(map(torch.Tensor.is_contiguous, tensors)):
            raise ValueError("%s: tensors must be contiguous" % what)
        return list(map(torch.Tensor.data_ptr, tensors))

    def _used_on(self, stream):
        """The states were made on the stream that was current at construction; the allocator has to know of this one."""
        for t in (self._progress, *self.state.values()):
            t.record_stream(stream)

    def step(self, grads=None, *, stream=None):
        """One step with the gradients given (fp32 or bf16, the parameters' shapes), by default each parameter's
        .grad; a parameter whose gradient is None is left out.  Returns the gradients' norm before clipping (a
        0-dim fp32 tensor on the device), or None without max_grad_norm."""
        lib = load()
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self.params):
            raise ValueError("%d gradients for %d parameters" % (len(grads), len(self.params)))
        table = self._table
        if list(map(_dtype, self.params)) != self._dtypes:
            raise TypeError("a parameter's dtype has changed")
        table["param"] = self._checked(self.params, "params")
        have = [g is not None for g in grads]
        if all(have):
            table["grad"] = self._checked(grads, "grads")
            dtypes = list(map(_dtype, grads))
            if dtypes != self._grad_dtypes:
                table["grad_dtype"] = [_io_dtype(g) for g in grads]
                self._grad_dtypes = dtypes
        else:
            if not any(have):
                return None
            table = table[have].copy()
            grads = [p if g is None else g for p, g in zip(self.params, grads)]
            table["grad"] = np.array(self._checked(grads, "grads"), np.uint64)[have]
            table["grad_dtype"] = np.array([_io_dtype(g) for g in grads])[have]
        if not (0 <= self.betas[0] < 1 and 0 <= self.betas[1] < 1 and 1e-30 <= self.eps <= 1e30
                and math.isfinite(self.lr) and math.isfinite(self.weight_decay)
                and (self.max_grad_norm is None or self.max_grad_norm > 0)):
            raise ValueError("lr %r, betas %r, eps %r, weight_decay %r, max_grad_norm %r: out of range"
                             % (self.lr, self.betas, self.eps, self.weight_decay, self.max_grad_norm))
        rows, count = ctypes.addressof(ctypes.c_char.from_buffer(table)), len(table)
        s, st, norm = _stream(stream, self.device), self.state, None
        get = st.get
        states = (_address(st["exp_avg"]), _address(st["exp_avg_sq"]), _address(get("exp_avg_base")),
                  _address(get("exp_avg_sq_base")), _address(get("master")))
        cfg = ssm_adamw_config(self.lr, self.betas[0], self.betas[1], self.eps, self.weight_decay, 0,
                               self.seed & (2 ** 64 - 1), self.state_bits, 0)
        if self.max_grad_norm is not None:
            if self._count is not None:
                if _capturing(stream):
                    raise RuntimeError("the steps so far were counted on the host: make one step with max_grad_norm "
                                       "before the capture")
                self._count_on_device(stream)
            norm = _empty((), torch.float32, self.device, stream)
            need = int(lib.ssm_grad_norm_workspace_size(rows, count))
            workspace = _empty(need, torch.uint8, self.device, stream)
            _check(lib.ssm_adamw_clipped_step(ctypes.byref(cfg), rows, count, float(self.max_grad_norm), *states,
                                              _address(self._progress), _address(norm), _address(workspace), need, s))
        else:
            if _capturing(stream):
                raise RuntimeError("without max_grad_norm every replay would repeat this step's number: set it "
                                   "(math.inf: no clipping) for steps in a graph")
            if self._count is None:
                self._count = self.step_count
            cfg.step = self._count + 1
            _check(lib.ssm_adamw_step(ctypes.byref(cfg), rows, count, *states, None, s))
            self._count += 1
        # a graph that has kept a parameter for its backward pass must be refused from now on
        increment_version(self.params if all(have) else [p for p, h in zip(self.params, have) if h])
        if stream is not None:
            self._used_on(stream)
            _hand_out(stream, norm)
        return norm

    def state_values(self, *, stream=None):
        """(m, v) of all tensors, flat, at their offsets: fp32 buffers as they are, 8-bit states as the values they
        stand for, in bf16 (exact)."""
        st = self.state
        if self.state_bits == 32:
            return st["exp_avg"], st["exp_avg_sq"]
        m = _empty(self.numel, torch.bfloat16, self.device, stream)
        v = _empty(self.numel, torch.bfloat16, self.device, stream)
        _check(load().ssm_adamw_state_values(self.numel, _address(st["exp_avg"]), _address(st["exp_avg_sq"]),
                                             _address(st["exp_avg_base"]), _address(st["exp_avg_sq_base"]), _address(m),
                                             _address(v), _stream(stream, self.device)))
        if stream is not None:
            self._used_on(stream)
            _hand_out(stream, m, v)
        return m, v
