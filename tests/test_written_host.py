"""What the kernels write into a caller's own tensors is told to autograd (without a GPU: the library is replaced): an operation
that has kept such a tensor for its backward pass must be refused, not go on with other values."""
import pytest
import torch

import selective_state_space_76_amd as ssm
from selective_state_space_76_amd import _lib as L
from selective_state_space_76_amd import block as K
from selective_state_space_76_amd import training as T

F32 = torch.float32
B, D, N, S, E, V = 2, 3, 4, 70, 5, 9


class Library:
    """Every size is 4096 bytes, a row has 7 checkpoints, every call succeeds."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("_size") else 7 if name.endswith("_checkpoints") else 0


@pytest.fixture
def plain(monkeypatch):
    for m in (L, T, K):
        monkeypatch.setattr(m, "load", Library)
        monkeypatch.setattr(m, "_ptr", lambda t: None)
        monkeypatch.setattr(m, "_stream", lambda stream, device: 0)
    for m in (T, K):
        monkeypatch.setattr(m, "_address", lambda t: None)


def t(*shape):
    return torch.zeros(shape)


U, ROW, STATE, BC, A = t(B, D, S), t(B, D), t(B, D, N), t(B, N, S), t(D, N)
TOK, TABLE, CH = torch.zeros(B, S, dtype=torch.int64), t(V, E), t(D)


def norm_grads(**g):
    return ssm.layer_norm_bwd(t(B, S, E), t(B, S, E), t(E), t(2, B * S), residual=True, p=0.5, seed=1, grads=g)


# name -> (call with the tensors by name, their shapes)
CALLS = {
    "scan": (lambda **k: ssm.scan_fwd(U, U, A, BC, BC, **k),
             dict(out=(B, D, S), final_state=(B, D, N), checkpoints=(B, 2, D, N))),
    "scan without a workspace": (lambda **k: ssm.scan_fwd_noalloc(U, U, A, BC, BC, **k),
                                 dict(out=(B, D, S), final_state=(B, D, N))),
    "scan gradients": (lambda **g: ssm.scan_bwd(U, U, A, BC, BC, None, U, dout=U, grads=g),
                       dict(du=(B, D, S), ddelta=(B, D, S), dA=(D, N), dB=(B, N, S), dC=(B, N, S), dD=(D,), dz=(B, D, S),
                            ddelta_bias=(D,), dinitial_state=(B, D, N))),
    "state update": (lambda state, **k: ssm.state_update(state, ROW, ROW, A, t(B, N), t(B, N), **k),
                     dict(state=(B, D, N), out=(B, D))),
    "conv": (lambda **k: ssm.conv1d_fwd(U, A, **k), dict(out=(B, D, S), final_state=(B, D, N - 1))),
    "conv step": (lambda state, **k: ssm.conv1d_update(state, ROW, A, **k), dict(state=(B, D, N - 1), out=(B, D))),
    "conv gradients": (lambda **g: ssm.conv1d_bwd(U, A, dout=U, grads=g),
                       dict(dx=(B, D, S), dweight=(D, N), dbias=(D,), dinitial_state=(B, D, N - 1))),
    "embedding": (lambda **k: ssm.embedding_fwd(TOK, TABLE, **k), dict(out=(B, S, E))),
    "embedding gradient": (lambda **k: ssm.embedding_bwd(TOK, t(B, S, E), V, **k), dict(dweight=(V, E))),
    "embedding gradient, added": (lambda **k: ssm.embedding_bwd(TOK, t(B, S, E), V, accumulate=True, **k), dict(dweight=(V, E))),
    "norm": (lambda **k: ssm.layer_norm_fwd(t(B, S, E), t(E), None, t(B, S, E), **k),
             dict(out=(B, S, E), hidden=(B, S, E), stats=(2, B * S))),
    "norm gradients": (norm_grads, dict(dx=(B, S, E), dresidual=(B, S, E), dweight=(E,), dbias=(E,))),
    "dropout": (lambda **k: ssm.dropout_fwd(U, 0.0, 1, **k), dict(out=(B, D, S))),
    "dropout gradient": (lambda **k: ssm.dropout_bwd(U, 0.0, 1, **k), dict(dx=(B, D, S))),
    "recurrence": (lambda **k: ssm.recurrence_fwd(U, U, U, CH, **k),
                   dict(out=(B, D, S), final_state=(B, D), checkpoints=(B, D, 7))),
    "recurrence gradients": (lambda **g: ssm.recurrence_bwd(U, U, U, CH, None, None, U, dout=U, grads=g),
                             dict(dx=(B, D, S), dr=(B, D, S), di=(B, D, S), dz=(B, D, S), ddecay=(D,), dr_bias=(D,),
                                  di_bias=(D,), dinitial_state=(B, D))),
    "recurrence step": (lambda state, **k: ssm.recurrence_update(state, ROW, ROW, ROW, CH, **k),
                        dict(state=(B, D), out=(B, D))),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_what_is_written_is_told(plain, monkeypatch, name):
    call, shapes = CALLS[name]
    monkeypatch.setattr(K, "_capturing", lambda stream: False)
    before = {id(x): x._version for x in (U, ROW, STATE, BC, A, TOK, TABLE, CH)}
    given = {k: torch.zeros(s) for k, s in shapes.items()}
    versions = {k: x._version for k, x in given.items()}
    call(**given)
    assert all(x._version > versions[k] for k, x in given.items()), name
    # and each alone, the others being made by the call
    for k in given:
        if name != "scan without a workspace" and not (k != "state" and "state" in given):
            x = torch.zeros(shapes[k])
            call(**{k: x})
            assert x._version == 1, (name, k)
    assert all(x._version == before[id(x)] for x in (U, ROW, STATE, BC, A, TOK, TABLE, CH))


def test_a_state_that_was_kept_is_refused(plain):
    """A loss of a recurrent state behind which another step is taken in place."""
    w = torch.ones(B, D, requires_grad=True)
    for step, state in ((lambda s: ssm.recurrence_update(s, ROW, ROW, ROW, CH), torch.ones(B, D)),
                        (lambda s: ssm.state_update(s, ROW, ROW, A, t(B, N), t(B, N)), torch.ones(B, D, N)),
                        (lambda s: ssm.conv1d_update(s, ROW, A), torch.ones(B, D, N - 1))):
        loss = (w.view(B, D, *[1] * (state.dim() - 2)) * state).sum()
        step(state)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
