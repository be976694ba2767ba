"""stream=: what the binding allocates belongs to the stream that the kernels run on (without a GPU: the allocations and
the streams they are made on are recorded)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import selective_state_space_76_amd as ssm
from selective_state_space_76_amd import _lib as L
from selective_state_space_76_amd import training as T

F32 = torch.float32


class Library:
    """Every size is 4096 bytes, every call succeeds."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("_size") else 0


@pytest.fixture
def record(monkeypatch):
    """(stream, address) of every allocation and of every tensor that the allocator is told of."""
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
    monkeypatch.setattr(torch, "empty_like", lambda t: allocate(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: r.current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: r.told.append((s, t.data_ptr())))
    for m in (L, T):
        monkeypatch.setattr(m, "load", Library)
        monkeypatch.setattr(m, "_ptr", lambda t: None)
    monkeypatch.setattr(T, "_address", lambda t: None)
    return r


u = torch.zeros(2, 3, 70)
A, BC, W4 = torch.zeros(3, 4), torch.zeros(2, 4, 70), torch.zeros(3, 4)
TOK, TABLE = torch.zeros(2, 70, dtype=torch.int64), torch.zeros(9, 3)


def step(**k):
    opt = ssm.AdamW([torch.zeros(300)], max_grad_norm=1.0, state_bits=8)
    opt.device = SimpleNamespace(index=-1)
    return opt, opt.step([torch.zeros(300)], **k)


def values(**k):
    opt = ssm.AdamW([torch.zeros(300)], state_bits=8)
    opt.device = SimpleNamespace(index=-1)
    return opt, opt.state_values(**k)


CALLS = {
    "scan": lambda **k: ssm.scan_fwd(u, u, A, BC, BC, **k),
    "scan gradients": lambda **k: ssm.scan_bwd(u, u, A, BC, BC, dout=u, **k),
    "state update": lambda **k: ssm.state_update(torch.zeros(2, 3, 4), u[..., 0], u[..., 0], A, BC[..., 0], BC[..., 0], **k),
    "conv": lambda **k: ssm.conv1d_fwd(u, W4, **k),
    "conv step": lambda **k: ssm.conv1d_update(u[..., :3], u[..., 0], W4, **k),
    "conv gradients": lambda **k: ssm.conv1d_bwd(u, W4, dout=u, **k),
    "embedding": lambda **k: ssm.embedding_fwd(TOK, TABLE, **k),
    "embedding gradient": lambda **k: ssm.embedding_bwd(TOK, torch.zeros(2, 70, 3), 9, **k),
    "optimizer step": step,
    "optimizer states": values,
}


def tensors(x):
    if isinstance(x, torch.Tensor):
        return [x]
    if isinstance(x, ssm.AdamW):
        return []
    return [t for y in (x.values() if isinstance(x, dict) else x) if y is not None for t in tensors(y)]


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_stream_of_the_call(record, name):
    side = SimpleNamespace(cuda_stream=7, device="cuda:0")
    out = CALLS[name](stream=side)
    # memory of the caller's stream may still be in use by what is queued there
    assert record.made and all(s is side for s, _ in record.made)
    # what the caller gets, it uses on its own stream
    returned = {t.data_ptr() for t in tensors(out)}
    assert returned <= {p for s, p in record.told if s == "callers"}
    if isinstance(out[0] if isinstance(out, tuple) else None, ssm.AdamW):  # made at construction, on the caller's stream
        assert {t.data_ptr() for t in out[0].state.values()} <= {p for s, p in record.told if s is side}


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_nothing_is_recorded(record, monkeypatch, name):
    monkeypatch.setattr(T, "_stream", lambda stream, device: 0)
    monkeypatch.setattr(L, "_stream", lambda stream, device: 0)
    CALLS[name]()
    assert record.made and all(s == "callers" for s, _ in record.made) and not record.told
