"""The residual block's operators without a GPU: every bad argument is refused on the host, by the C entry points and by
the binding; the mask's generator against the published vectors."""
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import selective_state_space_76_amd as ssm
from selective_state_space_76_amd import _lib as L
from selective_state_space_76_amd import block as K
from tests import block_ref as R

BASE = 1 << 40  # fake, aligned, never dereferenced


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 34) + off)


def drop(**kw):
    d = dict(p=0.1, seed=1, device_seed=None, call=0)
    d.update(kw)
    return L.ssm_dropout(*[d[k] for k in ("p", "seed", "device_seed", "call")])


def ref(s):
    return None if s is None else ctypes.byref(s)


def test_generator_gives_the_published_vectors():
    """The known answers that were published with the generator."""
    for c, k, want in (([0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
                       ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
                       ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
                        "d16cfe09 94fdcceb 5001e420 24126ea1")):
        assert " ".join("%08x" % w for w in R.philox(c, k)) == want
    seed, call = 0x299F31D0A4093822, 0x0370734413198A2E
    words = R.philox([5, 0, call & 0xFFFFFFFF, call >> 32], [seed & 0xFFFFFFFF, seed >> 32])
    halves = [h for w in words for h in (w & 0xFFFF, w >> 16)]
    for p in (0.25, 0.5):
        assert R.mask(8, p, seed, call, first=40)[0].tolist() == [h >= 65536 * p for h in halves]


def test_dropout_refusals():
    lib = L.load()

    def call(n=1000, xd=1, od=0, x=fake(1), res=fake(2), d=drop(), out=fake(3)):
        return lib.ssm_dropout_fwd(n, xd, od, x, res, ref(d), out, None)

    assert call(xd=2) == 3 and call(od=-1) == 3 and call(n=0) == 2 and call(n=-5) == 2 and call(n=1 << 43) == 2
    assert call(x=None) == 1 and call(out=None) == 1 and call(d=None) == 1
    for p in (-0.1, 1.5, float("nan"), float("inf")):
        assert call(d=drop(p=p)) == 5
    for k in ("x", "res", "out"):
        assert call(**{k: fake(7, 8)}) == 4
    assert call(d=drop(device_seed=fake(8, 4).value)) == 4
    assert call(out=fake(1, 512)) == 8 and call(out=fake(2)) == 8 and call(d=drop(device_seed=fake(3, 64).value)) == 8


def nshape(**kw):
    d = dict(batch=4, seqlen=50, dim=96, x_dtype=1, hidden_dtype=0, flags=0)
    d.update(kw)
    return L.ssm_norm_shape(*[d[k] for k, _ in L.ssm_norm_shape._fields_])


def test_layer_norm_refusals():
    lib = L.load()

    def fwd(s=nshape(), x=fake(1), w=fake(2), b=fake(3), res=fake(4), eps=1e-5, d=None, out=fake(5), hid=fake(6),
            stats=fake(7)):
        return lib.ssm_layer_norm_fwd(ref(s), x, w, b, res, eps, ref(d), out, hid, stats, None)

    def bwd(s=nshape(), dout=fake(1), hid=fake(2), w=fake(3), stats=fake(4), dh=fake(5), d=None, dx=fake(6), dr=fake(7),
            dw=fake(8), db=fake(9), work=fake(10), ws=1 << 30):
        return lib.ssm_layer_norm_bwd(ref(s), dout, hid, w, stats, dh, ref(d), dx, dr, dw, db, work, ws, None)

    for f in (fwd, bwd):
        assert f(s=None) == 1
        for bad in (dict(batch=0), dict(seqlen=0), dict(dim=0), dict(dim=(1 << 30) + 1), dict(batch=1 << 20, seqlen=1 << 12)):
            assert f(s=nshape(**bad)) == 2, bad
        for bad in (dict(x_dtype=2), dict(hidden_dtype=-1), dict(x_dtype=0, hidden_dtype=1)):
            assert f(s=nshape(**bad)) == 3, bad
        assert f(s=nshape(flags=2)) == 5 and f(s=nshape(flags=8)) == 5 and f(d=drop(p=2.0)) == 5
    for k in ("x", "out"):
        assert fwd(**{k: None}) == 1
    for eps in (-1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == 5
    for k in ("x", "w", "b", "res", "out", "hid"):
        assert fwd(**{k: fake(11, 8)}) == 4, k
    assert fwd(stats=fake(11, 2)) == 4
    assert fwd(out=fake(1)) == 8 and fwd(hid=fake(4)) == 8 and fwd(hid=fake(5, 32)) == 8 and fwd(stats=fake(5, 64)) == 8
    for k in ("dout", "hid", "stats", "work"):
        assert bwd(**{k: None}) == 1, k
    assert bwd(dx=None, dr=None) == 1
    for k in ("dout", "hid", "w", "dh", "dx", "dr", "dw", "db", "work"):
        assert bwd(**{k: fake(11, 4)}) == 4, k
    for flags in (0, 1):
        need = lib.ssm_layer_norm_bwd_workspace_size(ref(nshape(flags=flags)))
        assert need and need % (2 * 96 * 4) == 0 and bwd(s=nshape(flags=flags), ws=need - 1) == 6
    assert lib.ssm_layer_norm_bwd_workspace_size(ref(nshape(dim=0))) == 0
    assert bwd(dx=fake(1)) == 8 and bwd(dr=fake(2)) == 8 and bwd(dw=fake(9)) == 8 and bwd(work=fake(5, 16)) == 8
    assert bwd(db=fake(4, 32)) == 8 and bwd(work=fake(6, 16)) == 8


def rshape(**kw):
    d = dict(batch=2, dim=64, seqlen=1000, io_dtype=1, flags=0)
    d.update(kw)
    return L.ssm_recurrence_shape(*[d[k] for k, _ in L.ssm_recurrence_shape._fields_])


def test_recurrence_refusals():
    lib = L.load()

    def fwd(s=rshape(), x=fake(1), r=fake(2), i=fake(3), dec=fake(4), rb=None, ib=None, z=None, init=None, out=fake(5),
            last=fake(6), ck=fake(7), work=fake(8), ws=1 << 30):
        return lib.ssm_recurrence_fwd(ref(s), x, r, i, dec, rb, ib, z, init, out, last, ck, work, ws, None)

    def bwd(s=rshape(), x=fake(1), r=fake(2), i=fake(3), dec=fake(4), rb=None, ib=None, z=None, init=None, dout=fake(5),
            dl=None, ck=None, dx=fake(6), dr=fake(7), di=fake(8), dz=None, dd=fake(9), drb=fake(10), dib=fake(11), d0=fake(12),
            work=fake(13), ws=1 << 30):
        return lib.ssm_recurrence_bwd(ref(s), x, r, i, dec, rb, ib, z, init, dout, dl, ck, dx, dr, di, dz, dd, drb, dib, d0,
                                      work, ws, None)

    for f in (fwd, bwd):
        assert f(s=None) == 1
        for bad in (dict(batch=0), dict(dim=0), dict(seqlen=0), dict(batch=1 << 16, dim=1 << 16), dict(seqlen=1 << 41)):
            assert f(s=rshape(**bad)) == 2, bad
        assert f(s=rshape(io_dtype=2)) == 3 and f(s=rshape(flags=1)) == 5 and f(s=rshape(flags=4)) == 5
        for k in ("x", "r", "i", "dec"):
            assert f(**{k: None}) == 1 and f(**{k: fake(14, 8)}) == 4, k
    need = lib.ssm_recurrence_workspace_size(ref(rshape(seqlen=100000)))
    assert need and fwd(s=rshape(seqlen=100000), ws=need - 1) == 6 and fwd(s=rshape(seqlen=100000), work=None) == 1
    assert lib.ssm_recurrence_workspace_size(ref(rshape(dim=0))) == 0 == lib.ssm_recurrence_checkpoints(ref(rshape(flags=1)))
    for k in ("rb", "ib", "z", "init", "last", "ck", "work"):
        assert fwd(**{k: fake(14, 8)}) == 4, k
    assert fwd(out=None) == 1 and fwd(out=fake(2)) == 8 and fwd(last=fake(4)) == 8 and fwd(ck=fake(5, 64)) == 8
    for k in ("dout", "dx", "dr", "di", "dd", "work"):
        assert bwd(**{k: None}) == 1, k
    assert bwd(z=fake(14)) == 1
    for k in ("dout", "dl", "ck", "dx", "dr", "di", "dd", "drb", "dib", "d0", "work"):
        assert bwd(**{k: fake(14, 8)}) == 4, k
    for ck in (None, fake(14)):
        need = lib.ssm_recurrence_bwd_workspace_size(ref(rshape()), 0 if ck is None else 1)
        assert bwd(ck=ck, ws=need - 1) == 6
    assert bwd(dx=fake(1)) == 8 and bwd(dr=fake(6, 64)) == 8 and bwd(dd=fake(4)) == 8 and bwd(work=fake(3, 32)) == 8
    assert bwd(z=fake(14), dz=fake(14)) == 8

    def step(B=4, D=30, io=1, st=fake(1), x=fake(2), r=fake(3), i=fake(4), dec=fake(5), rb=None, ib=None, z=None, out=fake(6)):
        return lib.ssm_recurrence_update(B, D, io, st, x, r, i, dec, rb, ib, z, out, None)

    assert step(B=0) == 2 and step(D=-1) == 2 and step(io=5) == 3
    for k in ("st", "x", "r", "i", "dec", "out"):
        assert step(**{k: None}) == 1 and step(**{k: fake(14, 4)}) == 4, k
    assert step(out=fake(2)) == 8 and step(st=fake(3)) == 8 and step(out=fake(1, 16)) == 8


def test_checkpoints_cover_every_row():
    """One for every 64 pieces, the pieces that a row of odd length shares with its neighbours included."""
    for B, D, n in ((1, 1, 1), (2, 3, 511), (2, 3, 512), (1, 5, 513), (3, 7, 4099)):
        for io, v in ((1, 8), (0, 4)):
            blocks = ssm.recurrence_checkpoints_shape(B, D, n, io)[2]
            row = np.arange(B * D)
            assert blocks * 64 * v >= n + max(row * n % v) and (blocks - 1) * 64 * v < n + v


def test_binding_refusals():
    x = torch.zeros(2, 3, 8)
    w = torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        ssm.layer_norm_fwd(x, w)
    with pytest.raises(ValueError, match="residual: expected shape"):
        ssm.layer_norm_fwd(x, w, None, x[:1])
    with pytest.raises(TypeError, match="residual and hidden"):
        ssm.layer_norm_fwd(x, w, None, x.bfloat16())
    with pytest.raises(ValueError, match="weight: expected shape"):
        ssm.layer_norm_fwd(x, w, channels_first=True)
    with pytest.raises(ValueError, match="channels_first"):
        ssm.layer_norm_fwd(x[0], w, channels_first=True)
    with pytest.raises(TypeError, match="weight"):
        ssm.layer_norm_fwd(x, w.bfloat16())
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.layer_norm_fwd(x.half(), w)
    with pytest.raises(ValueError, match="rows=0"):
        ssm.layer_norm_fwd(x[:0], w)
    with pytest.raises(ValueError, match="no dimension"):
        ssm.layer_norm_fwd(torch.zeros(()), w)
    with pytest.raises(ValueError, match="seqlen=0"):
        ssm.layer_norm_fwd(x[:, :, :0], w, channels_first=True)
    with pytest.raises(ValueError, match="x itself"):
        ssm.layer_norm_fwd(x, w, hidden=x)
    for p in (-0.5, 1.01, float("nan")):
        with pytest.raises(ValueError, match="p must be"):
            ssm.dropout_fwd(x, p, 1)
    with pytest.raises(ValueError, match="seed"):
        ssm.layer_norm_fwd(x, w, p=0.1)
    with pytest.raises(TypeError, match="seed"):
        ssm.dropout_fwd(x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError, match="seed"):
        ssm.dropout_fwd(x, 0.1, torch.zeros(1))
    with pytest.raises(ValueError, match="numel=0"):
        ssm.dropout_bwd(x[:0], 0.1, 1)
    stats = torch.zeros(2, 6)
    with pytest.raises(ValueError, match="stats: expected shape"):
        ssm.layer_norm_bwd(x, x, w, stats[:, :5])
    with pytest.raises(TypeError, match="x's dtype"):
        ssm.layer_norm_bwd(x, x, w, stats, x_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dresidual is not computed"):
        ssm.layer_norm_bwd(x, x, w, stats, grads={"dresidual": x.clone()})
    d = torch.zeros(3)
    with pytest.raises(ValueError, match="r: expected shape"):
        ssm.recurrence_fwd(x, x[:, :, :4], x, d)
    with pytest.raises(ValueError, match="GPU"):
        ssm.recurrence_fwd(x, x, x, d)
    with pytest.raises(ValueError, match="decay"):
        ssm.recurrence_fwd(x, x, x, torch.zeros(4))
    with pytest.raises(ValueError, match="checkpoints: expected shape"):
        ssm.recurrence_bwd(x, x, x, d, dout=x, checkpoints=torch.zeros(2, 3, 2))
    with pytest.raises(ValueError, match="seqlen=0"):
        ssm.recurrence_fwd(x[:, :, :0], x[:, :, :0], x[:, :, :0], d)
    with pytest.raises(ValueError, match=r"\[B, D\]"):
        ssm.recurrence_update(torch.zeros(2, 3), x, x, x, d)
    with pytest.raises(TypeError, match="state"):
        ssm.recurrence_update(torch.zeros(2, 3).bfloat16(), x[..., 0], x[..., 0], x[..., 0], d)


def test_a_mask_that_replays_would_repeat_is_refused(monkeypatch):
    monkeypatch.setattr(K, "_capturing", lambda stream: True)
    monkeypatch.setattr(K, "_ptr", lambda t: 0)
    x = torch.zeros(2, 8)
    for f in (lambda s: ssm.dropout_fwd(x, 0.1, s), lambda s: ssm.layer_norm_fwd(x, p=0.1, seed=s)):
        with pytest.raises(RuntimeError, match="repeat"):
            f(7)
    assert K._mask(0.1, torch.zeros(1, dtype=torch.int64), 0, x.device, None, True) is not None
    assert K._mask(0.1, 7, 0, x.device, None, False) is not None  # a backward pass takes its forward pass's mask
    assert K._mask(0.0, None, 0, x.device, None, True) is None


def test_seeds_are_integers_of_any_kind():
    """numpy's, too, and negative ones: the same 64 bits; nothing that is no integer."""
    for seed, call in ((-5, 3), (2 ** 63 + 1, 2 ** 64 - 1), (np.int64(-5), np.int32(3)), (np.uint64(2 ** 63 + 1), np.int64(-1))):
        m = K._mask(0.5, seed, call, torch.device("cpu"), None, False)
        assert (m.seed, m.call) == (int(seed) % 2 ** 64, int(call) % 2 ** 64)
    for seed in (1.5, "7"):
        with pytest.raises(TypeError):
            K._mask(0.5, seed, 0, torch.device("cpu"), None, False)


class Library:
    """Every size is 4096 bytes, every call succeeds."""

    def __getattr__(self, name):
        return lambda *args: 2 if name.endswith("checkpoints") else 4096 if name.endswith("_size") else 0


x3, d3, s3 = torch.zeros(2, 3, 700), torch.zeros(3), torch.zeros(2, 3)
CALLS = {
    "norm": lambda **k: ssm.layer_norm_fwd(x3, torch.zeros(700), None, x3, p=0.5, seed=1, **k),
    "norm gradients": lambda **k: ssm.layer_norm_bwd(x3, x3, torch.zeros(700), torch.zeros(2, 6), residual=True, **k),
    "dropout": lambda **k: ssm.dropout_fwd(x3, 0.5, 1, **k),
    "dropout gradient": lambda **k: ssm.dropout_bwd(x3, 0.5, 1, **k),
    "recurrence": lambda **k: ssm.recurrence_fwd(x3, x3, x3, d3, **k),
    "recurrence gradients": lambda **k: ssm.recurrence_bwd(x3, x3, x3, d3, dout=x3, **k),
    "recurrence step": lambda **k: ssm.recurrence_update(s3, x3[..., 0], x3[..., 0], x3[..., 0], d3, **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_stream_of_the_call(monkeypatch, name):
    """What the binding allocates belongs to the stream that the kernels run on; what is returned is the caller's."""
    import contextlib
    r = SimpleNamespace(current="callers", made=[], told=[])

    @contextlib.contextmanager
    def on(stream):
        before, r.current = r.current, stream
        yield
        r.current = before

    empty = torch.empty

    def allocate(*a, device=None, **k):
        t = empty(*a, **k)
        r.made.append((r.current, t.data_ptr()))
        return t

    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: allocate(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: r.current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: r.told.append((s, t.data_ptr())))
    monkeypatch.setattr(K, "load", Library)
    monkeypatch.setattr(K, "_address", lambda t: None)
    monkeypatch.setattr(K, "_arg", lambda *a: None if a[0] is None else 0)
    monkeypatch.setattr(K, "_capturing", lambda stream: False)
    monkeypatch.setattr(K, "_stream", lambda stream, device: 0)
    side = SimpleNamespace(cuda_stream=7, device="cuda:0")
    out = CALLS[name](stream=side)
    returned = [t for t in (out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else [out])
                if t is not None]
    assert r.made and all(s is side for s, _ in r.made)
    assert {t.data_ptr() for t in returned} <= {p for s, p in r.told if s == "callers"}
    r.made, r.told = [], []
    CALLS[name]()
    assert r.made and all(s == "callers" for s, _ in r.made) and not r.told
