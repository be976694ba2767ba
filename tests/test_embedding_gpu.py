"""The embedding and its gradient (GPU) against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from selective_state_space_76_amd import embedding, embedding_bwd, embedding_fwd
from tests.train_ref import embed_grad, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def tokens_of(B, L, V, seed, kind="mixed", dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "mixed":  # frequent low tokens, and marks outside the table
        t = ((V + 1) ** torch.rand(B, L, generator=g, dtype=torch.float64) - 1).long().clamp_(0, V - 1)
        u = torch.rand(B, L, generator=g)
        t[u < 0.1] = -1
        t[(u >= 0.1) & (u < 0.13)] = V
        t[(u >= 0.13) & (u < 0.15)] = 2 ** 31 - 1 if dtype == torch.int32 else 2 ** 40
    elif kind == "same":
        t = torch.full((B, L), V - 1)
    elif kind == "none":
        t = torch.full((B, L), -1)
    else:
        t = torch.randint(0, V, (B, L), generator=g)
    return t.to(dtype)


def fwd_ref(tok, w, scale, dtype, cf):
    ok = (tok >= 0) & (tok < w.shape[0])
    r = torch.where(ok[..., None], w[tok.long().clamp(0, w.shape[0] - 1)].float() * scale, 0.0).to(dtype)
    return r.transpose(1, 2).contiguous() if cf else r


@pytest.mark.parametrize("wt", [F32, BF16], ids=["wf32", "wbf16"])
@pytest.mark.parametrize("ot", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("cf", [False, True], ids=["ble", "bel"])
@pytest.mark.parametrize("B,L,V,E", [(1, 1, 1, 1), (2, 3, 5, 7), (3, 130, 11, 64), (2, 257, 1000, 72), (1, 128, 4, 128),
                                     (5, 61, 300, 193)])
def test_forward(wt, ot, cf, B, L, V, E):
    print("case: embed", wt, ot, cf, B, L, V, E, flush=True)
    tok = tokens_of(B, L, V, seed=B * L + E)
    w = torch.randn(V, E, generator=torch.Generator().manual_seed(E)).to(wt)
    for scale in (1.0, 27.712812921102035):
        out = embedding_fwd(tok.to(DEV), w.to(DEV), scale=scale, dtype=ot, channels_first=cf)
        assert torch.equal(out.cpu(), fwd_ref(tok, w, float(np.float32(scale)), ot, cf))  # one rounding: the same bits


def test_forward_int32_step_and_special_values():
    w = torch.randn(50, 40)
    w[3, 5], w[4, 6], w[5, 0] = float("nan"), float("inf"), -0.0
    tok = tokens_of(1, 64, 50, seed=3, dtype=torch.int32).reshape(-1)  # one token for each of 64 sequences
    out = embedding_fwd(tok.to(DEV), w.to(DEV)).cpu()
    assert out.shape == (64, 40)
    assert torch.equal(torch.nan_to_num(out, 7.0), torch.nan_to_num(fwd_ref(tok, w, 1.0, F32, False), 7.0))
    into = torch.full((64, 40), 9.0, dtype=BF16, device=DEV)
    assert embedding_fwd(tok.to(DEV), w.to(DEV), out=into) is into
    assert torch.equal(torch.nan_to_num(into.cpu(), 7.0), torch.nan_to_num(fwd_ref(tok, w, 1.0, BF16, False), 7.0))


def bwd_check(tok, V, E, ot, gt, cf, scale, seed, add=False):
    B, L = tok.shape
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(B * L, E, generator=g).to(ot)
    t = tok.reshape(-1)
    outside = (t < 0) | (t >= V)
    rows[outside] = float("nan")  # what a masked position holds must not matter
    d = rows.reshape(B, L, E)
    d = d.transpose(1, 2).contiguous() if cf else d
    old = torch.randn(V, E, generator=g).to(gt) if add else None
    dw = embedding_bwd(tok.to(DEV), d.to(DEV), V, scale=scale, channels_first=cf, dtype=gt,
                       dweight=None if old is None else old.to(DEV), accumulate=add)
    ref, mag, n = embed_grad(t.numpy(), f64(rows), V, scale)
    if add:
        ref = ref + f64(old)
    got = f64(dw)
    # n terms added in fp32 in some order: at most n units in the last place of their magnitudes' sum, and the product
    # with the scale; a bf16 result is rounded once more
    tol = (n[:, None] + 3) * 2.0 ** -24 * (mag + (np.abs(f64(old)) if add else 0))
    if gt == BF16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref)[bad].max()))
    if add:
        idle = n == 0
        assert torch.equal(dw.cpu()[torch.from_numpy(idle)], old[torch.from_numpy(idle)])
    return dw


@pytest.mark.parametrize("ot", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gt", [F32, BF16], ids=["gf32", "gbf16"])
@pytest.mark.parametrize("cf", [False, True], ids=["ble", "bel"])
@pytest.mark.parametrize("B,L,V,E", [(1, 1, 1, 1), (2, 3, 5, 7), (1, 31, 3, 8), (2, 16, 4, 64), (1, 33, 700, 260),
                                     (3, 130, 11, 64), (2, 257, 255, 72), (2, 300, 256, 512), (5, 461, 3000, 193)])
def test_backward(ot, gt, cf, B, L, V, E):
    for k, kind in enumerate(("mixed", "same", "none", "even")):
        print("case: embed grad", ot, gt, cf, B, L, V, E, kind, flush=True)
        bwd_check(tokens_of(B, L, V, B * L + E, kind), V, E, ot, gt, cf, 1.0 if k % 2 else 1.7, seed=E + k)
    bwd_check(tokens_of(B, L, V, 1, "mixed", torch.int32), V, E, ot, gt, cf, 0.5, seed=2, add=True)


@pytest.mark.parametrize("V", [1, 2, 4, 15, 16, 17, 31, 32, 33, 63, 64, 65, 300])
@pytest.mark.parametrize("ot", [F32, BF16], ids=["f32", "bf16"])
def test_backward_few_rows_channels_first(V, ot):
    """The scan's layout with a small alphabet: ragged ends of positions and channels, several batch rows."""
    for B, L, E in ((1, 2100, 40), (3, 1029, 130), (2, 4096, 16)):
        print("case: embed grad letters", V, ot, B, L, E, flush=True)
        for add in (False, True):
            bwd_check(tokens_of(B, L, V, V + L), V, E, ot, F32, True, 2.5, seed=V, add=add)


@pytest.mark.parametrize("V,cf", [(4, True), (40, True), (4, False), (300, True)])
@pytest.mark.parametrize("ot", [F32, BF16], ids=["f32", "bf16"])
def test_infinite_and_nan_gradients_stay_with_their_token(V, cf, ot):
    """A value that is not finite reaches its own token's row and channel and no other."""
    B, L, E = 2, 1500, 70
    tok = tokens_of(B, L, V, V)
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(B, L, E, generator=g).to(ot)
    tok[0, 7], tok[1, 1490], tok[1, 1499] = 1, 2, 0
    rows[(tok < 0) | (tok >= V)] = float("inf")
    rows[0, 7, 5], rows[1, 1490, 69], rows[1, 1499, 0] = float("nan"), float("inf"), -float("inf")
    d = rows.transpose(1, 2).contiguous() if cf else rows
    got = f64(embedding_bwd(tok.to(DEV), d.to(DEV), V, channels_first=cf))
    with np.errstate(invalid="ignore"):
        ref, mag, n = embed_grad(tok.reshape(-1).numpy(), f64(rows).reshape(-1, E), V, 1.0)
    assert np.isnan(got[1, 5]) and got[2, 69] == np.inf and got[0, 0] == -np.inf
    fine = np.isfinite(ref)
    assert fine.sum() == fine.size - 3 and np.isfinite(got[fine]).all()
    assert (np.abs(got - ref)[fine] <= ((n[:, None] + 3) * 2.0 ** -24 * mag)[fine]).all()


# more than one tile of the sort, one to three digits, and chunks of every length
@pytest.mark.parametrize("n,V,E", [(8192, 50000, 8), (8193, 70000, 8), (9000, 255, 24), (20001, 256, 16),
                                   (66000, 3, 8), (66001, 20, 8), (300007, 70001, 4), (600011, 5, 4)])
@pytest.mark.parametrize("kind", ["mixed", "same"])
def test_backward_sort_sizes(n, V, E, kind):
    print("case: embed grad of", n, V, E, kind, flush=True)
    bwd_check(tokens_of(1, n, V, n, kind), V, E, F32, F32, False, 1.0, seed=n)


# short lists: one launch or several by what is to be cleared, how wide the rows are and where 1024, 2048 and 4096 end
@pytest.mark.parametrize("n,V,E", [(17, 50000, 20), (1000, 4096, 260), (1023, 4097, 260), (1024, 1 << 20, 4),
                                   (1025, 700, 24), (2500, 50000, 24), (4096, 300, 24), (1024, 40, 4096),
                                   (2047, 16384, 260), (2048, 16385, 24), (2049, 5000, 260), (1500, 50, 2000),
                                   (1024, 40, 4100), (700, 9, 2600)])
@pytest.mark.parametrize("add", [False, True], ids=["new", "added"])
def test_backward_short_lists(n, V, E, add):
    for kind in ("mixed", "same", "even", "none"):
        print("case: embed grad of", n, V, E, add, kind, flush=True)
        dw = bwd_check(tokens_of(1, n, V, n + E, kind), V, E, BF16 if E > 24 else F32, F32, False, 1.5, seed=n, add=add)
        if kind == "none" and not add:
            assert not dw.any()


def test_backward_is_the_transpose():
    """<dout, embed(W + D) - embed(W)> = <gradient, D>: the map is linear, so differences are exact but for rounding."""
    V, E = 90, 50
    tok = tokens_of(2, 200, V, 5)
    D = torch.randn(V, E)
    dout = torch.randn(2, 200, E)
    dw = embedding_bwd(tok.to(DEV), dout.to(DEV), V, scale=3.0)
    a = float((f64(embedding_fwd(tok.to(DEV), D.to(DEV), scale=3.0)) * f64(dout)).sum())
    b = float((f64(dw) * f64(D)).sum())
    assert abs(a - b) <= 1e-5 * float(np.abs(f64(dw) * f64(D)).sum())


def test_autograd_and_same_bits():
    V, E = 333, 96
    tok = tokens_of(4, 700, V, 6).to(DEV)
    dout = torch.randn(4, E, 700, device=DEV).to(BF16)
    grads = []
    for _ in range(2):
        w = torch.randn(V, E, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV).requires_grad_(True)
        embedding(tok, w, scale=2.0, channels_first=True).backward(dout)
        grads.append(w.grad)
    want = embedding_bwd(tok, dout, V, scale=2.0, channels_first=True, dtype=BF16)
    assert grads[0].dtype == BF16 and torch.equal(grads[0], grads[1]) and torch.equal(grads[0], want)


def test_another_stream():
    V, E = 1000, 256
    tok, dout = tokens_of(2, 5000, V, 9).to(DEV), torch.randn(2, 5000, E, device=DEV)
    a = embedding_bwd(tok, dout, V)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = embedding_bwd(tok, dout, V, stream=side)
    c = embedding_fwd(tok, a, stream=side)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(c, embedding_fwd(tok, a))


@pytest.mark.parametrize("cf,V", [(False, 1000), (True, 1000), (True, 5)], ids=["ble", "bel", "bel-letters"])
def test_more_than_2_31_elements(cf, V):
    T, E = (1 << 21) + 3, 1030
    print("case: embed %d x %d" % (T, E), cf, V, flush=True)
    tok = tokens_of(1, T, V, 4, "even").to(DEV)
    w = torch.randn(V, E, device=DEV).to(BF16)
    out = embedding_fwd(tok, w, channels_first=cf)
    rows = out[0].t() if cf else out[0]
    for lo in (0, T // 2, T - 200):
        assert torch.equal(rows[lo:lo + 200], w[tok[0, lo:lo + 200]])
    # the gradient of out's own values: every row of the table times its count
    dw = embedding_bwd(tok, out, V, channels_first=cf)
    n = torch.bincount(tok[0], minlength=V).double()[:, None]
    ref = w.double() * n
    assert bool(((dw.double() - ref).abs() <= (n + 2) * 2.0 ** -24 * ref.abs()).all())
