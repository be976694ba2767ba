"""Calls for tensors of another device than the current one (without a GPU: the library, the devices and their streams are
replaced): the library is called while the tensors' device is the current one, since a default stream is known by its
device only; a stream of another device is refused."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import selective_state_space_76_amd as ssm
from selective_state_space_76_amd import _lib as L
from selective_state_space_76_amd import block as K
from selective_state_space_76_amd import training as T

HERE, THERE = torch.device("cuda:0"), torch.device("cuda:1")


class There(torch.Tensor):
    """A tensor that says it is on the second device."""
    device = property(lambda self: THERE)


@pytest.fixture
def two(monkeypatch):
    """The current device is the first; .calls: (entry point, the device that was current)."""
    r = SimpleNamespace(now=0, calls=[])

    class Library:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 4096
            if name.endswith("_checkpoints"):
                return lambda *a: 7
            return lambda *a: r.calls.append((name, r.now)) or 0

    @contextlib.contextmanager
    def on(index):
        before, r.now = r.now, index if isinstance(index, int) else index.index
        yield
        r.now = before

    empty = torch.empty
    there = lambda *a, device=None, **k: empty(*a, **k).as_subclass(There)  # noqa: E731
    monkeypatch.setattr(torch, "empty", there)
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: there(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: r.now, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", on)
    stream = lambda d=0: SimpleNamespace(cuda_stream=0, device=torch.device("cuda", d) if isinstance(d, int) else d)  # noqa: E731
    monkeypatch.setattr(torch.cuda, "current_stream", stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext() if s is None else on(s.device))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: r.now == 1)  # only the second device's is
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    for m in (L, T, K):
        monkeypatch.setattr(m, "load", Library)
        monkeypatch.setattr(m, "_ptr", lambda t: None)
    for m in (T, K):
        monkeypatch.setattr(m, "_address", lambda t: None)
    return r


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(There)


B, D, N, S = 2, 3, 4, 70


def adamw(bits, clip, **k):
    opt = ssm.AdamW([torch.zeros(300)], state_bits=bits, max_grad_norm=clip)
    opt.device = THERE
    opt.step([torch.zeros(300)], **k)


def values(**k):
    opt = ssm.AdamW([torch.zeros(300)], state_bits=8)
    opt.device = THERE
    opt.state_values(**k)


def calls():
    u, row, bc, a, ch, tok = t(B, D, S), t(B, D), t(B, N, S), t(D, N), t(D), t(B, S, dtype=torch.int64)
    return {
        "scan": lambda **k: ssm.scan_fwd(u, u, a, bc, bc, **k),
        "scan, saved": lambda **k: ssm.scan_fwd(u, u, a, bc, bc, checkpoints=t(B, 2, D, N), **k),
        "scan without a workspace": lambda **k: ssm.scan_fwd_noalloc(u, u, a, bc, bc, out=t(B, D, S), **k),
        "scan gradients": lambda **k: ssm.scan_bwd(u, u, a, bc, bc, dout=u, **k),
        "scan gradients, saved": lambda **k: ssm.scan_bwd(u, u, a, bc, bc, dout=u, checkpoints=t(B, 2, D, N), **k),
        "state update": lambda **k: ssm.state_update(t(B, D, N), row, row, a, t(B, N), t(B, N), **k),
        "conv": lambda **k: ssm.conv1d_fwd(u, a, **k),
        "conv step": lambda **k: ssm.conv1d_update(t(B, D, N - 1), row, a, **k),
        "conv gradients": lambda **k: ssm.conv1d_bwd(u, a, dout=u, **k),
        "embedding": lambda **k: ssm.embedding_fwd(tok, t(9, 5), **k),
        "embedding gradient": lambda **k: ssm.embedding_bwd(tok, t(B, S, 5), 9, **k),
        "norm": lambda **k: ssm.layer_norm_fwd(u, t(S), None, u, **k),
        "norm gradients": lambda **k: ssm.layer_norm_bwd(u, u, t(S), t(2, B * D), **k),
        "dropout": lambda **k: ssm.dropout_fwd(u, 0.5, t(1, dtype=torch.int64), **k),
        "dropout gradient": lambda **k: ssm.dropout_bwd(u, 0.5, 1, **k),
        "recurrence": lambda **k: ssm.recurrence_fwd(u, u, u, ch, **k),
        "recurrence gradients": lambda **k: ssm.recurrence_bwd(u, u, u, ch, dout=u, **k),
        "recurrence step": lambda **k: ssm.recurrence_update(t(B, D), row, row, row, ch, **k),
        "optimizer step, clipped": lambda **k: adamw(8, 1.0, **k),
        "optimizer states": values,
    }


@pytest.mark.parametrize("name", list(calls()))
def test_the_library_is_called_on_the_tensors_device(two, name):
    calls()[name]()
    assert two.calls and all(where == 1 for _, where in two.calls) and two.now == 0, two.calls


@pytest.mark.parametrize("name", list(calls()))
def test_a_stream_of_another_device_is_refused(two, name):
    with pytest.raises(ValueError, match="stream: expected one of cuda:1, got one of cuda:0"):
        calls()[name](stream=SimpleNamespace(cuda_stream=5, device=HERE))
    assert not two.calls and two.now == 0
    calls()[name](stream=SimpleNamespace(cuda_stream=5, device=THERE))
    assert two.calls and all(where == 1 for _, where in two.calls)


def test_the_capture_of_the_tensors_device_counts(two):
    """With a seed that every replay would repeat; steps whose number it would."""
    with pytest.raises(RuntimeError, match="every replay would repeat"):
        ssm.dropout_fwd(t(B, D), 0.5, 1)
    with pytest.raises(RuntimeError, match="every replay would repeat"):
        adamw(32, None)
    assert not two.calls


def test_no_device_is_changed_on_the_current_one(two, monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", None)
    two.now = 1
    ssm.recurrence_update(t(B, D), t(B, D), t(B, D), t(B, D), t(D))
    assert two.calls == [("ssm_recurrence_update", 1)]
