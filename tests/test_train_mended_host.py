"""The training operators without a GPU: what a call must refuse, plan or pass on."""
import copy
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from selective_state_space_76_amd import _lib as L
from selective_state_space_76_amd import training as T
from tests.test_train_host import cfg, fake, rows

OVERLAP, LAUNCH = 8, 7


def step(t):
    """The status of a step: LAUNCH where every check passed (there is no GPU here)."""
    return L.load().ssm_adamw_step(ctypes.byref(cfg()), t.ctypes.data, len(t), fake(1), fake(2), None, None, None, None, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would run on made-up addresses")
@pytest.mark.parametrize("count", [2, 3, 100, 2048, 2049, 5000])
def test_adamw_refuses_a_param_over_any_gradient_or_param(count):
    """Workgroups of one tensor would write what those of another read."""
    base = fake(3).value
    order = np.random.default_rng(count).permutation(2 * count) * 1024  # params and gradients in no order, side by side

    def make(**at):
        t = rows(*[dict(param=base + int(order[2 * k]), grad=base + int(order[2 * k + 1]), numel=512, offset=512 * k)
                   for k in range(count)])
        for k, (name, v) in at.items():
            t[name][int(k[1:])] = v
        return t

    good = make()
    assert step(good) == LAUNCH  # they touch, they do not overlap
    first, last = 0, count - 1
    for a, b in ((first, last), (last, first), (last, last)):
        for off in (0, 1008, -1008):
            assert step(make(**{"k%d" % a: ("grad", int(good["param"][b]) + off)})) == OVERLAP, (a, b, off)
    for off in (0, 1008, -1008):
        assert step(make(**{"k%d" % last: ("param", int(good["param"][first]) + off)})) == OVERLAP
    # two tensors with one gradient: nothing is written there
    assert step(make(**{"k%d" % last: ("grad", int(good["grad"][first]))})) == LAUNCH


@pytest.mark.parametrize("B,Ln,V,E", [(8192, 16, 64, 1024), (65536, 2, 64, 1024), (1 << 20, 3, 60, 64), (4096, 64, 4, 1024),
                                      (100000, 17, 32, 300), (1024, 255, 64, 1024), (64, 2, 64, 256), (1, 1 << 20, 4, 1024)])
@pytest.mark.parametrize("io", [0, 1], ids=["f32", "bf16"])
def test_embedding_gradient_workspace_of_many_short_rows(B, Ln, V, E, io):
    """What is kept beside dout is no more than a turned copy of it, the sorted lists (16 bytes a position and their sums)
    and a few MB, whatever the lengths of the batch rows."""
    s = L.ssm_embed_shape(batch=B, seqlen=Ln, rows=V, dim=E, index_dtype=1, table_dtype=0, io_dtype=io, flags=1)
    dout = B * Ln * E * (2 if io else 4)
    need = L.load().ssm_embedding_bwd_workspace_size(ctypes.byref(s))
    assert 0 < need <= 1.5 * dout + 32 * B * Ln + (8 << 20)


class Library:
    """Every size is 4096 bytes, every call succeeds and does nothing."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("_size") else 0


@pytest.fixture
def unplugged(monkeypatch):
    """The binding on CPU tensors, without the library."""
    for m in (L, T):
        monkeypatch.setattr(m, "load", Library)
        monkeypatch.setattr(m, "_ptr", lambda t: None)
        monkeypatch.setattr(m, "_stream", lambda stream, device: 0)
    monkeypatch.setattr(T, "_address", lambda t: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))

    def make(params, **k):
        opt = T.AdamW(params, **k)
        opt.device = SimpleNamespace(index=-1)
        return opt

    return make


@pytest.mark.parametrize("clip", [None, 1.0])
def test_a_step_is_an_in_place_change(unplugged, clip):
    """A graph built before the step must not be run on the changed weights in silence."""
    p, q = (torch.ones(300, requires_grad=True) for _ in range(2))
    opt = unplugged([p, q], max_grad_norm=clip)
    loss = (p * p).sum()
    other = (q * q).sum()
    p.grad = torch.ones(300)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    other.backward()  # without a gradient it was left out, and is what it was
    opt.step([torch.ones(300)] * 2)
    assert (p._version, q._version) == (2, 1)


def clipped(t=None, c=None, max_norm=1.0, count=None, m=fake(1), v=fake(2), mb=None, vb=None, master=None, progress=fake(3),
            norm=fake(4), work=fake(5), ws=1 << 20):
    t = rows({}, {}) if t is None else t
    return L.load().ssm_adamw_clipped_step(ctypes.byref(c or cfg()), t.ctypes.data, len(t) if count is None else count,
                                           max_norm, m, v, mb, vb, master, progress, norm, work, ws, None)


def test_clipped_step_refusals():
    good = rows({}, {})
    assert L.load().ssm_adamw_clipped_step(None, good.ctypes.data, 2, 1.0, fake(1), fake(2), None, None, None, fake(3),
                                           fake(4), fake(5), 1 << 20, None) == 1
    for k in ("m", "v", "progress", "norm", "work"):
        assert clipped(**{k: None}) == 1, k
    assert clipped(c=cfg(state_bits=8)) == 1 and clipped(rows(dict(grad=0))) == 1 and clipped(rows(dict(param=0))) == 1
    assert clipped(count=0) == 2 and clipped(rows(dict(numel=0))) == 2 and clipped(rows({}, dict(offset=256))) == 2
    assert clipped(rows(dict(param_dtype=2))) == 3 and clipped(rows(dict(grad_dtype=-1))) == 3
    for k in ("m", "v", "master", "progress", "work"):
        assert clipped(**{k: fake(6, 8)}) == 4, k
    assert clipped(norm=fake(4, 2)) == 4 and clipped(rows(dict(grad=fake(11).value + 8))) == 4
    for bad in (dict(state_bits=16), dict(flags=1), dict(lr=float("nan")), dict(beta1=1.0), dict(eps=0.0)):
        assert clipped(c=cfg(**bad)) == 5, bad
    assert clipped(max_norm=0.0) == 5 and clipped(max_norm=float("nan")) == 5
    need = L.load().ssm_grad_norm_workspace_size(good.ctypes.data, 2)
    assert clipped(ws=need - 1) == 6
    for k, off in (("progress", 16), ("norm", 4), ("work", 16)):
        for at in (1, 2, 10, 11, 12):  # the states, a param, its gradient, the next param
            assert clipped(**{k: fake(at, off)}) == OVERLAP, (k, at)
        assert clipped(**{k: fake(6, off), "master": fake(6)}) == OVERLAP
    assert clipped(norm=fake(3, 28)) == OVERLAP and clipped(norm=fake(5, 12)) == OVERLAP
    assert clipped(progress=fake(5)) == OVERLAP and clipped(rows(dict(grad=fake(10).value))) == OVERLAP


def test_where_the_step_is_counted(unplugged):
    """On the host without max_grad_norm; with it the host does not know, and what it knew is passed on once."""
    p, g = [torch.ones(300)], [torch.ones(300)]
    opt = unplugged(p, step=7)
    opt.step(g)
    assert opt._count == 8 == opt.step_count
    opt.max_grad_norm = 1.0
    opt.step(g)
    assert opt._count is None and int(opt._progress[0]) == 8  # (the library, which counts it, is not there)
    opt = unplugged(p, step=7, max_grad_norm=1.0)
    assert opt._count is None and int(opt._progress[0]) == 7
    opt._progress[0] = 5  # two of its steps were left out
    opt.max_grad_norm = None
    opt._count = 5  # (read from the device, for which there has to be one)
    opt.step(g)
    assert opt.step_count == 6


def test_a_capture_that_would_repeat_a_step_is_refused(unplugged, monkeypatch):
    p, g = [torch.ones(300)], [torch.ones(300)]
    opt, clips = unplugged(p), unplugged(p, max_grad_norm=1.0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="repeat this step's number"):
        opt.step(g)
    opt.max_grad_norm = 1.0
    with pytest.raises(RuntimeError, match="before the capture"):
        opt.step(g)
    assert opt.step_count == 0 and p[0]._version == 0
    clips.step(g)


def test_alignment_is_looked_at_when_the_optimizer_is_made(unplugged):
    with pytest.raises(L.SSMError, match="ALIGN.*a parameter"):
        unplugged([torch.zeros(64), torch.zeros(65)[1:]])
    with pytest.raises(L.SSMError, match="ALIGN.*exp_avg_sq"):
        unplugged([torch.zeros(128)], state={"exp_avg_sq": torch.zeros(129)[1:]})
    unplugged([torch.zeros(64), torch.zeros(68)[4:]])


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would run on made-up addresses")
@pytest.mark.parametrize("index,size", [(0, 4), (1, 8)], ids=["int32", "int64"])
def test_tokens_need_their_own_alignment_only(index, size):
    """A micro-batch is a row of a batch: with an odd length it begins off 16 bytes."""
    s = L.ssm_embed_shape(batch=1, seqlen=509, rows=1000, dim=64, index_dtype=index, table_dtype=0, io_dtype=1, flags=0)
    lib = L.load()
    for off in range(0, 16, 2):
        want = LAUNCH if off % size == 0 else 4
        assert lib.ssm_embedding_fwd(ctypes.byref(s), fake(1, off), fake(2), 1.0, fake(3), None) == want
        assert lib.ssm_embedding_bwd(ctypes.byref(s), fake(1, off), fake(2), 1.0, fake(3), fake(4), 1 << 30, None) == want


def test_a_copied_optimizer_has_a_table_of_its_own(unplugged, monkeypatch):
    seen = []

    class Looks(Library):
        def __getattr__(self, name):
            if name == "ssm_adamw_step":
                return lambda cfg, rows, count, *a: seen.append((rows, ctypes.c_uint64.from_address(rows).value)) or 0
            return Library.__getattr__(self, name)

    monkeypatch.setattr(T, "load", Looks)
    opt = unplugged([torch.ones(300)])
    twin = copy.deepcopy(opt)
    for o in (opt, twin):
        o.step([torch.ones(300)])
        assert seen[-1] == (o._table.ctypes.data, o.params[0].data_ptr())
    assert seen[0][0] != seen[1][0]
