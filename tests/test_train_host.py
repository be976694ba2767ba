"""The training operators without a GPU: every bad argument is refused on the host, by the C entry points
and by the binding."""
import ctypes

import numpy as np
import pytest
import torch

from selective_state_space_76_amd import AdamW, conv1d_bwd, embedding_bwd, embedding_fwd
from selective_state_space_76_amd import _lib as L
from selective_state_space_76_amd import training as T

BASE = 1 << 40  # fake, aligned, never dereferenced


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 34) + off)


def conv(lib, sizes=(2, 64, 100, 4), io=1, ws=1 << 30, **kw):
    a = dict(x=fake(1), w=fake(2), b=None, init=None, dout=fake(3), dfin=None, dx=fake(4), dw=fake(5), db=fake(6),
             dinit=None, work=fake(7))
    a.update(kw)
    return lib.ssm_conv1d_bwd(*sizes, io, *[a[k] for k in ("x", "w", "b", "init", "dout", "dfin", "dx", "dw", "db", "dinit",
                                                             "work")], ws, None)


def test_conv_bwd_refusals():
    lib = L.load()
    for k in ("x", "w", "dout", "dx", "dw", "work"):
        assert conv(lib, **{k: None}) == 1, k
    for sizes in ((0, 64, 100, 4), (2, 0, 100, 4), (2, 64, 0, 4), (2, 64, 100, 0), (2, 64, 100, 5), (1 << 41, 1, 1, 1),
                  (1 << 20, 1 << 20, 1, 4)):
        assert conv(lib, sizes) == 2, sizes
    assert conv(lib, io=2) == 3
    for k in ("x", "w", "b", "init", "dout", "dfin", "dx", "dw", "db", "dinit", "work"):
        assert conv(lib, **{k: fake(9, 8)}) == 4, k
    need = lib.ssm_conv1d_bwd_workspace_size(2, 64, 100, 4, 1)
    assert need == 2 * 64 * 5 * 4
    assert conv(lib, ws=need - 1) == 6
    assert conv(lib, dx=fake(1)) == 8 and conv(lib, dw=fake(3, 64)) == 8 and conv(lib, db=fake(4, 128)) == 8
    assert conv(lib, work=fake(1, 16)) == 8 and conv(lib, init=fake(4, 32)) == 8 and conv(lib, dinit=fake(3)) == 8
    # a window of one step has no state: its pointers are ignored
    assert lib.ssm_conv1d_bwd_workspace_size(0, 64, 100, 4, 1) == 0 == lib.ssm_conv1d_bwd_workspace_size(2, 64, 100, 4, 5)


def eshape(**kw):
    d = dict(batch=2, seqlen=50, rows=1000, dim=64, index_dtype=1, table_dtype=0, io_dtype=1, flags=0)
    d.update(kw)
    return L.ssm_embed_shape(**d)


def test_embedding_refusals():
    lib = L.load()

    def fwd(s=None, tok=fake(1), w=fake(2), out=fake(3), scale=1.0):
        return lib.ssm_embedding_fwd(ctypes.byref(s or eshape()), tok, w, scale, out, None)

    def bwd(s=None, tok=fake(1), d=fake(2), dw=fake(3), work=fake(4), ws=1 << 30, scale=1.0):
        return lib.ssm_embedding_bwd(ctypes.byref(s or eshape()), tok, d, scale, dw, work, ws, None)

    assert lib.ssm_embedding_fwd(None, fake(1), fake(2), 1.0, fake(3), None) == 1
    for k in ("tok", "w", "out"):
        assert fwd(**{k: None}) == 1 and fwd(**{k: fake(5, 4)}) == 4, k
    for k in ("tok", "d", "dw", "work"):
        assert bwd(**{k: None}) == 1 and bwd(**{k: fake(5, 4)}) == 4, k
    for f in (fwd, bwd):
        for bad in (dict(batch=0), dict(seqlen=0), dict(rows=0), dict(dim=0), dict(batch=1 << 16, seqlen=1 << 16),
                    dict(rows=1 << 31), dict(dim=1 << 41), dict(seqlen=1 << 30, dim=1 << 12)):
            assert f(eshape(**bad)) == 2, bad
        for bad in (dict(index_dtype=2), dict(table_dtype=-1), dict(io_dtype=7)):
            assert f(eshape(**bad)) == 3, bad
        assert f(eshape(flags=4)) == 5
        assert f(scale=float("nan")) == 5 and f(scale=float("inf")) == 5
    assert fwd(eshape(flags=2)) == 5  # adding is the gradient's
    assert fwd(out=fake(2, 1024)) == 8 and fwd(out=fake(1)) == 8
    assert bwd(dw=fake(2, 64)) == 8 and bwd(work=fake(3)) == 8 and bwd(dw=fake(1)) == 8
    need = lib.ssm_embedding_bwd_workspace_size(ctypes.byref(eshape()))
    assert need > 0 and bwd(ws=need - 1) == 6
    assert lib.ssm_embedding_bwd_workspace_size(ctypes.byref(eshape(dim=0))) == 0


def rows(*tensors):
    t = np.zeros(len(tensors), T._TENSOR)
    for k, d in enumerate(tensors):
        base = dict(param=fake(10 + 2 * k).value, grad=fake(11 + 2 * k).value, numel=300, offset=384 * k, param_dtype=1,
                    grad_dtype=1)
        base.update(d)
        for name, v in base.items():
            t[name][k] = v
    return t


def cfg(**kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, seed=0, state_bits=32, flags=0)
    d.update(kw)
    return L.ssm_adamw_config(*[d[k] for k, _ in L.ssm_adamw_config._fields_])


def test_adamw_refusals():
    lib = L.load()

    def step(t=None, c=None, count=None, m=fake(1), v=fake(2), mb=None, vb=None, master=None, clip=None):
        t = rows({}, {}) if t is None else t
        return lib.ssm_adamw_step(ctypes.byref(c or cfg()), t.ctypes.data, len(t) if count is None else count, m, v, mb, vb,
                                  master, clip, None)

    good = rows({}, {})
    assert lib.ssm_adamw_step(None, good.ctypes.data, 2, fake(1), fake(2), None, None, None, None, None) == 1
    assert lib.ssm_adamw_step(ctypes.byref(cfg()), None, 2, fake(1), fake(2), None, None, None, None, None) == 1
    assert step(m=None) == 1 and step(v=None) == 1 and step(c=cfg(state_bits=8)) == 1
    assert step(rows({}, dict(param=0))) == 1 and step(rows(dict(grad=0))) == 1
    assert step(count=0) == 2 and step(rows(dict(numel=0))) == 2 and step(rows({}, dict(offset=256))) == 2
    assert step(rows({}, dict(offset=385))) == 2 and step(rows(dict(offset=-128))) == 2
    assert step(rows(dict(param_dtype=2))) == 3 and step(rows(dict(grad_dtype=-1))) == 3
    assert step(rows(dict(param=fake(10).value + 2))) == 4 and step(rows(dict(grad=fake(11).value + 8))) == 4
    for k in ("m", "v", "master"):
        assert step(**{k: fake(3, 8)}) == 4
    assert step(clip=fake(3, 2)) == 4
    for bad in (dict(state_bits=16), dict(flags=1), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0),
                dict(step=0), dict(weight_decay=float("inf"))):
        assert step(c=cfg(**bad)) == 5, bad
    assert step(v=fake(1, 1024)) == 8 and step(m=fake(10)) == 8 and step(master=fake(11)) == 8
    assert step(rows(dict(grad=fake(10).value))) == 8 and step(clip=fake(1, 8)) == 8
    assert lib.ssm_grad_norm(good.ctypes.data, 2, 0.0, fake(1), fake(2), 1 << 20, None) == 5
    assert lib.ssm_grad_norm(good.ctypes.data, 2, 1.0, None, fake(2), 1 << 20, None) == 1
    need = lib.ssm_grad_norm_workspace_size(good.ctypes.data, 2)
    assert need == 16 and lib.ssm_grad_norm(good.ctypes.data, 2, 1.0, fake(1), fake(2), need - 1, None) == 6
    assert lib.ssm_grad_norm(good.ctypes.data, 2, 1.0, fake(11), fake(2), need, None) == 8
    assert lib.ssm_adamw_state_values(100, *[fake(k) for k in range(1, 7)], None) == 2
    assert lib.ssm_adamw_state_values(256, fake(1), fake(2), fake(3), fake(4), None, None, None) == 1
    assert lib.ssm_adamw_state_values(256, fake(1), fake(2), fake(3), None, fake(5), fake(6), None) == 1
    assert lib.ssm_adamw_state_values(256, fake(1), fake(2), fake(3), fake(4), fake(1), fake(6), None) == 8


def test_binding_refusals():
    x = torch.zeros(2, 3, 5)
    w = torch.zeros(3, 4)
    with pytest.raises(ValueError, match="GPU"):
        conv1d_bwd(x, w, dout=x)
    with pytest.raises(ValueError, match="dout: expected shape"):
        conv1d_bwd(x, w, dout=x[:, :, :4])
    with pytest.raises(TypeError, match="dout"):
        conv1d_bwd(x, w, dout=x.to(torch.bfloat16))
    with pytest.raises(ValueError, match="seqlen=0"):
        conv1d_bwd(x[:, :, :0], w, dout=x[:, :, :0])
    tok, table = torch.zeros(2, 5, dtype=torch.int64), torch.zeros(7, 3)
    with pytest.raises(TypeError, match="int32 or int64"):
        embedding_fwd(tok.float(), table)
    with pytest.raises(ValueError, match="channels_first"):
        embedding_fwd(tok[0], table, channels_first=True)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        embedding_fwd(tok, table.half())
    with pytest.raises(ValueError, match="seqlen=0"):
        embedding_fwd(tok[:, :0], table)
    for scale in (float("nan"), float("inf")):
        with pytest.raises(ValueError, match="scale"):
            embedding_fwd(tok, table, scale=scale)
        with pytest.raises(ValueError, match="scale"):
            embedding_bwd(tok, torch.zeros(2, 5, 3), 7, scale=scale)
    with pytest.raises(ValueError, match="GPU"):
        embedding_fwd(tok, table)
    with pytest.raises(ValueError, match="dout: expected shape"):
        embedding_bwd(tok, torch.zeros(2, 4, 3), 7)
    with pytest.raises(ValueError, match="dimensions"):
        embedding_bwd(tok, torch.zeros(10, 3), 7)
    with pytest.raises(ValueError, match="accumulate"):
        embedding_bwd(tok, torch.zeros(2, 5, 3), 7, accumulate=True)
    with pytest.raises(ValueError, match="rows=0"):
        embedding_bwd(tok, torch.zeros(2, 5, 3), 0)
    with pytest.raises(ValueError, match="no parameters"):
        AdamW([])
    with pytest.raises(ValueError, match="state_bits"):
        AdamW([table], state_bits=16)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        AdamW([table.half()])
    with pytest.raises(ValueError, match="GPU"):
        AdamW([table])
