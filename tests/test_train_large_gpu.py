"""The training operators (GPU) where a launch's workgroups go on in a second dimension: 2^32 threads and more."""
import ctypes

import pytest
import torch

from selective_state_space_76_amd import _lib as L
from selective_state_space_76_amd import conv1d_bwd, embedding_bwd, embedding_fwd
from tests.train_ref import conv_grads, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def free():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def rel(a, b):
    return float((abs(f64(a) - b) / (abs(b) + 1e-2)).max())


@pytest.mark.parametrize("B,D", [(1, (1 << 28) + 37), (2, (1 << 27) + 37)], ids=["one row", "two rows"])
def test_conv_gradients_of_2_28_rows(B, D):
    """One step of very many channels: 16 rows to a workgroup, and with two batch rows the join of their sums."""
    print("case: conv grad", B, D, flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    x, dout = (torch.empty(B, D, 1, dtype=BF16, device=DEV).normal_(generator=g) for _ in range(2))
    w = torch.randn(D, 2, generator=g, device=DEV)
    out = conv1d_bwd(x, w, dout=dout)
    for lo in (0, 1 << 22, D // 2 - 50, D - 100):
        s = slice(lo, lo + 100)
        ref = conv_grads(f64(x[:, s]), f64(w[s]), None, None, f64(dout[:, s]), None)
        for name, r, tol in zip(("dx", "dweight", "dbias", "dinitial_state"), ref, (1e-2, 1e-3, 1e-3, 1e-2)):
            assert rel(out[name][s] if name in ("dweight", "dbias") else out[name][:, s], r) <= tol, (name, lo)


def test_embedding_of_2_24_short_rows():
    """[B, E, L] with two positions a row: a tile each, forward and gradient."""
    B, E, V = (1 << 24) + 3, 32, 3
    print("case: embed", B, E, V, flush=True)
    g = torch.Generator(device=DEV).manual_seed(2)
    tok = torch.randint(-1, V, (B, 2), generator=g, device=DEV, dtype=torch.int32)
    w = torch.randn(V, E, generator=g, device=DEV).to(BF16)
    out = embedding_fwd(tok, w, channels_first=True)
    wide = torch.cat([w, torch.zeros_like(w[:1])])
    for lo in (0, 1 << 22, B // 2, B - 1000):
        assert torch.equal(out[lo:lo + 1000], wide[tok[lo:lo + 1000].long()].transpose(1, 2))
    dw = embedding_bwd(tok, out, V, channels_first=True)
    n = torch.bincount(tok.view(-1) + 1, minlength=V + 1)[1:].double()[:, None]
    ref = w.double() * n
    assert bool(((dw.double() - ref).abs() <= (n + 2) * 2.0 ** -24 * ref.abs()).all())


def test_embedding_of_2_35_elements():
    """[B, L, E]: 64 GiB."""
    T, E, V = (1 << 20) + 1, 1 << 15, 7
    print("case: embed", T, E, V, flush=True)
    g = torch.Generator(device=DEV).manual_seed(3)
    tok = torch.randint(0, V, (T,), generator=g, device=DEV)
    w = torch.randn(V, E, generator=g, device=DEV).to(BF16)
    out = embedding_fwd(tok, w)
    for lo in (0, 1 << 17, T // 2, T - 100):
        assert torch.equal(out[lo:lo + 100], w[tok[lo:lo + 100]])


@pytest.mark.parametrize("n", [100, 5000])
def test_gradient_of_a_table_of_64_gib(n):
    """What a sort's launches clear beside it, one launch or several."""
    V, E = (1 << 24) + 5, 1024
    print("case: embed grad of a large table", n, flush=True)
    g = torch.Generator(device=DEV).manual_seed(4)
    tok = torch.randperm(V, generator=g, device=DEV)[:n]
    dout = torch.randn(n, E, generator=g, device=DEV)
    dw = torch.empty(V, E, device=DEV)
    for part in dw.split(1 << 21):
        part.fill_(1.0)
    embedding_bwd(tok, dout, V, dweight=dw)
    assert torch.equal(dw[tok], dout)
    dw[tok] = 0.0
    assert not any(bool(part.any()) for part in dw.split(1 << 21))


def test_state_values_of_2_35_codes():
    n = (1 << 35) + 128
    print("case: states read out", n, flush=True)
    codes = torch.zeros(n, dtype=torch.uint8, device=DEV)
    base = torch.full((n // 128,), 889, dtype=torch.int16, device=DEV)
    out = torch.empty(n, dtype=BF16, device=DEV)
    for lo in (0, (1 << 33) - 1000, n - 1000):
        codes[lo:lo + 1000] = 127  # 127 + 889 = 8 * 127: one
    s = torch.cuda.current_stream().cuda_stream
    p = [None if t is None else ctypes.c_void_p(t.data_ptr()) for t in (codes, None, base, None, out, None)]
    assert L.load().ssm_adamw_state_values(n, *p, s) == 0
    torch.cuda.synchronize()
    for lo in (0, (1 << 33) - 1000, n - 1000):
        assert bool((out[lo:lo + 1000] == 1).all())
    assert sum(int(part.count_nonzero()) for part in out.split(1 << 32)) == 3000
