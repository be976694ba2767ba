"""Layer norm and RMS norm (GPU) against their 64-bit formulas and against differences.

Tolerances.  u = 2^-24.  A sum over E is taken by lanes of at most 64 terms each (E / 256 and a tree of 16 on the long
rows): off by N u times the sum of magnitudes, N = 80 + E / 256.  The mean is off by (N + 2) u mean|s|, the factor by
(N / 2 + 6) u of itself and what the mean's error does to the spread; out = (s - m) f w + b takes four more roundings, and
one to its type of at most half a step (finfo.eps / 2)."""
import numpy as np
import pytest
import torch

from selective_state_space_76_amd import layer_norm, layer_norm_bwd, layer_norm_bwd_workspace_size, layer_norm_fwd
from tests import block_ref as R
from tests.train_ref import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = R.U
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]
IDS = ["f32", "bf16", "bf16-f32"]


def half(dtype):
    return torch.finfo(dtype).eps / 2 if dtype != F32 else U


def rows_of(t, cf):
    """[rows, E] in 64 bits; None stays."""
    if t is None:
        return None
    a = f64(t)
    return np.moveaxis(a, 1, -1).reshape(-1, a.shape[1]) if cf else a.reshape(-1, a.shape[-1])


def make(shape, xt, ht, seed, cf=False, weight=True, bias=True, residual=True, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    E = shape[1] if cf else shape[-1]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(r(*shape) + shift).to(xt), weight=1 + 0.3 * r(E) if weight else None, bias=r(E) if bias else None,
                residual=(2 * r(*shape)).to(ht) if residual else None, dout=r(*shape).to(xt), dhidden=r(*shape).to(ht))


def gpu(t):
    return None if t is None else t.to(DEV)


def dropped(x, p, seed, call, cf):
    """(rows of dropout(x), what a rounding of the product may be off by)."""
    if p == 0.0:
        return rows_of(x, cf)
    a = R.drop(f64(x), p, seed, call)
    return np.moveaxis(a, 1, -1).reshape(-1, a.shape[1]) if cf else a.reshape(-1, a.shape[-1])


def check_fwd(i, eps=1e-5, rms=False, cf=False, p=0.0, seed=77, call=5):
    out, hidden, stats = layer_norm_fwd(gpu(i["x"]), gpu(i["weight"]), gpu(i["bias"]), gpu(i["residual"]), eps=eps, rms=rms,
                                        channels_first=cf, p=p, seed=seed, call=call)
    torch.cuda.synchronize()
    res = rows_of(i["residual"], cf)
    s = dropped(i["x"], p, seed, call, cf) + (0.0 if res is None else res)
    w = None if i["weight"] is None else f64(i["weight"])
    b = None if i["bias"] is None else f64(i["bias"])
    ref, _, m, f = R.norm_of(s, w, b, eps, rms)
    E = s.shape[1]
    N = 80 + E // 256
    mag = np.abs(s).mean(1)
    es = 2 * U * (np.abs(s) + (0 if res is None else np.abs(res)))  # of the sum itself: the product, the addition
    em = (0.0 if rms else (N + 2) * U * mag + es.mean(1)) * np.ones_like(mag)
    d = s - m[:, None]
    # the spread: each (s - m) off by es + em + u |s - m|; mean of 2 |d| of it, and the sum's own error
    var = (d * d).mean(1)
    ev = (2 * np.abs(d) * (es + em[:, None] + U * np.abs(d))).mean(1) + (em ** 2) + (N + 4) * U * var
    ef = (ev / (2 * (var + eps)) + 4 * U) * f
    ww = np.abs(1.0 if w is None else w)
    tol = ww * ((es + em[:, None] + U * np.abs(d)) * f[:, None] + np.abs(d) * ef[:, None]) + 4 * U * (
        np.abs(d * f[:, None]) * ww + np.abs(0.0 if b is None else b)) + half(out.dtype) * np.abs(ref) * (1 + 2 ** -6)
    got = rows_of(out, cf)
    assert (np.abs(got - ref) <= tol + 1e-37).all(), float((np.abs(got - ref) / (tol + 1e-37)).max())
    mean, factor = f64(stats)
    assert (np.abs(mean - m) <= em + U * np.abs(m)).all() and (np.abs(factor - f) <= ef + U * f).all()
    if i["residual"] is None and p == 0.0:
        assert hidden.data_ptr() != out.data_ptr() and torch.equal(hidden.cpu(), i["x"])
    else:
        assert hidden.dtype == (i["x"] if i["residual"] is None else i["residual"]).dtype
        assert (np.abs(rows_of(hidden, cf) - s) <= es + half(hidden.dtype) * np.abs(s) * (1 + 2 ** -6)).all()
    return out, hidden, stats


def check_bwd(i, rms=False, cf=False, p=0.0, seed=77, call=5, residual=True, eps=1e-5):
    """hidden: i's residual (or x)."""
    hid = i["residual"] if residual else i["x"]
    rows = rows_of(hid, cf)
    w = None if i["weight"] is None else f64(i["weight"])
    _, _, m, f = R.norm_of(rows, None, None, eps, rms)
    stats = torch.from_numpy(np.stack([m, f]).astype(np.float32))
    m, f = f64(stats)
    dh = i["dhidden"] if residual else None
    g = layer_norm_bwd(gpu(i["dout"]), gpu(hid), gpu(i["weight"]), gpu(stats), dhidden=gpu(dh), rms=rms, channels_first=cf,
                       p=p, seed=seed, call=call, residual=residual, bias=i["bias"] is not None)
    torch.cuda.synchronize()
    d, q = rows_of(i["dout"], cf), rows_of(dh, cf)
    ds, dw, db = R.norm_grads(d, rows, w, m, f, q, rms)
    E, n = rows.shape[1], rows.shape[0]
    N = 80 + E // 256
    xh = np.abs(rows - m[:, None]) * f[:, None]
    exh = 2 * U * xh + U * (np.abs(rows) + np.abs(m[:, None])) * f[:, None]
    gg = np.abs(d * (1.0 if w is None else w))
    c2 = (gg * xh).mean(1, keepdims=True)
    ec = ((N + 3) * U * gg.mean(1, keepdims=True) * (0 if rms else 1)
          + xh * ((N + 4) * U * c2 + (gg * exh).mean(1, keepdims=True)) + exh * c2)
    c1 = 0.0 if rms else gg.mean(1, keepdims=True)
    tol = f[:, None] * (ec + 4 * U * (gg + c1 + xh * c2)) + U * (np.abs(ds) + (0 if q is None else np.abs(q)))
    if residual:
        got = rows_of(g["dresidual"], cf)
        lim = tol + half(g["dresidual"].dtype) * np.abs(ds) * (1 + 2 ** -6) + 1e-37
        assert g["dresidual"].dtype == hid.dtype and (np.abs(got - ds) <= lim).all(), float((np.abs(got - ds) / lim).max())
    back = ds
    if p:
        full = i["dout"].shape
        B, E_, L = full if cf else (1, 1, 1)
        mem = np.moveaxis(ds.reshape(B, L, E_), -1, 1) if cf else ds.reshape(full)
        back = R.drop(np.ascontiguousarray(mem), p, seed, call)
        back = np.moveaxis(back, 1, -1).reshape(-1, E) if cf else back.reshape(-1, E)
    got = rows_of(g["dx"], cf)
    scale = 1 / (1 - p) * 1.001
    lim = tol * scale + U * np.abs(back) + half(g["dx"].dtype) * np.abs(back) * (1 + 2 ** -6) + 1e-37
    assert g["dx"].dtype == i["x"].dtype and (np.abs(got - back) <= lim).all(), float((np.abs(got - back) / lim).max())
    # sums over rows: a chain of every row at the most
    M = min(n, 64 + n // 64) + 64
    for got, want, parts, each in ((g["dweight"], dw, np.abs(d) * xh, np.abs(d) * exh), (g["dbias"], db, np.abs(d), 0 * d)):
        if got is not None:
            lim = (M + 2) * U * parts.sum(0) + each.sum(0) + U * np.abs(want)
            assert got.dtype == F32 and (np.abs(f64(got) - want) <= lim).all(), float((np.abs(f64(got) - want) / lim).max())
    assert (g["dweight"] is None) == (i["weight"] is None) and (g["dbias"] is None) == (i["bias"] is None)
    return g


# widths around a piece of 8, the lanes' and registers' limits, and odd ones
WIDTHS = [1, 7, 8, 9, 33, 64, 127, 128, 129, 256, 257, 511, 513, 768, 1000, 1024, 1025, 2048, 2056, 3333, 4096, 4104, 8192,
          8200, 16384, 16392, 40001]


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("E", WIDTHS)
def test_rows(types, E):
    print("case: norm rows", types, E, flush=True)
    rows = 37 if E < 2000 else 5
    i = make((rows, E), *types, seed=E)
    check_fwd(i)
    check_bwd(i)
    i = make((rows, E), *types, seed=E + 1, bias=False, residual=False)
    check_fwd(i, rms=True)
    if types[0] == types[1]:
        check_bwd(i, rms=True, residual=False)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("B,E,L", [(1, 1, 2), (2, 3, 7), (1, 16, 8), (3, 33, 63), (2, 64, 64), (2, 100, 65), (1, 128, 200),
                                   (2, 129, 31), (1, 300, 129), (1, 512, 128), (1, 513, 72), (2, 768, 96), (1, 1024, 257),
                                   (1, 1030, 64), (2, 2048, 40), (1, 2500, 33), (5, 40, 1), (1, 8200, 17)])
def test_channels_first(types, B, E, L):
    print("case: norm cols", types, B, E, L, flush=True)
    i = make((B, E, L), *types, seed=E + L, cf=True)
    check_fwd(i, cf=True)
    check_bwd(i, cf=True)
    i = make((B, E, L), *types, seed=E + L + 1, cf=True, bias=False, residual=False)
    check_fwd(i, rms=True, cf=True)
    if types[0] == types[1]:
        check_bwd(i, rms=True, cf=True, residual=False)


@pytest.mark.parametrize("cf", [False, True], ids=["rows", "cols"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("shape", [(3, 40, 24), (2, 77, 131), (1, 768, 64), (2, 1111, 50)])
def test_dropout_inside(types, cf, shape):
    print("case: norm with dropout", types, cf, shape, flush=True)
    i = make(shape, *types, seed=sum(shape), cf=cf)
    for p in (0.1, 0.5, 1.0):
        check_fwd(i, cf=cf, p=p, seed=(9 << 40) + 3, call=1 << 33)
        if p < 1:
            check_bwd(i, cf=cf, p=p, seed=(9 << 40) + 3, call=1 << 33)
    alone = dict(i, residual=None)
    check_fwd(alone, cf=cf, p=0.3)


@pytest.mark.parametrize("cf", [False, True], ids=["rows", "cols"])
def test_layouts_of_one_step_agree(cf):
    """[B, E, 1] is [B, 1, E]."""
    i = make((6, 200, 1), BF16, F32, seed=3, cf=True)
    a = layer_norm_fwd(gpu(i["x"]), gpu(i["weight"]), gpu(i["bias"]), gpu(i["residual"]), channels_first=True)
    b = layer_norm_fwd(gpu(i["x"][..., 0]), gpu(i["weight"]), gpu(i["bias"]), gpu(i["residual"][..., 0]))
    assert torch.equal(a[0][..., 0], b[0]) and torch.equal(a[1][..., 0], b[1]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("cf", [False, True], ids=["rows", "cols"])
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_far_from_zero_and_constant_rows(rms, cf):
    """A large common part: the spread is taken about the mean.  A row without spread: the bias, whatever the row."""
    shape = (2, 384, 40) if cf else (80, 384)
    check_fwd(make(shape, F32, F32, seed=4, cf=cf, residual=False, shift=3000.0), rms=rms, cf=cf)
    i = make(shape, F32, F32, seed=5, cf=cf, residual=False)
    i["x"].fill_(2.5)
    out, _, stats = check_fwd(i, rms=rms, cf=cf)
    if not rms:
        want = i["bias"].view((-1, 1) if cf else (-1,)).expand(shape)
        assert torch.equal(out.cpu(), want) and torch.equal(stats[0].cpu(), torch.full((80,), 2.5))
    i["x"].zero_()
    check_fwd(i, rms=rms, cf=cf)


@pytest.mark.parametrize("cf", [False, True], ids=["rows", "cols"])
def test_what_is_not_finite_stays_in_its_row(cf):
    """Infinities and NaN spoil their own row alone; a dropped one does not even that."""
    shape = (2, 96, 70) if cf else (140, 96)
    i = make(shape, BF16, BF16, seed=6, cf=cf)
    bad = i["x"].clone()
    view = bad.transpose(1, 2).reshape(140, 96) if cf else bad
    view = view.clone()
    view[3, 5], view[77, 0], view[139, 95] = float("inf"), float("nan"), -float("inf")
    bad = (view.reshape(2, 70, 96).transpose(1, 2) if cf else view).contiguous()
    args = [gpu(i[k]) for k in ("weight", "bias", "residual")]
    good = layer_norm_fwd(gpu(i["x"]), *args, channels_first=cf)[0]
    got = layer_norm_fwd(gpu(bad), *args, channels_first=cf)[0]
    a, b = (torch.from_numpy(rows_of(t, cf)) for t in (good, got))
    fine = torch.tensor([k not in (3, 77, 139) for k in range(140)])
    assert torch.equal(a[fine], b[fine]) and torch.isnan(b[~fine]).any(1).all()
    assert torch.isfinite(layer_norm_fwd(gpu(bad), *args, channels_first=cf, p=1.0, seed=1)[0]).all()


@pytest.mark.parametrize("cf", [False, True], ids=["rows", "cols"])
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_against_differences(rms, cf):
    """<grad, direction> against central differences of the 64-bit form, dropout and the hidden output included."""
    shape = (2, 48, 9) if cf else (3, 6, 48)
    i = make(shape, F32, F32, seed=8, cf=cf)
    p, seed, call = 0.4, 12345, 3
    out, hidden, stats = layer_norm_fwd(*[gpu(i[k]) for k in ("x", "weight", "bias", "residual")], rms=rms,
                                        channels_first=cf, p=p, seed=seed, call=call)
    g = layer_norm_bwd(gpu(i["dout"]), hidden, gpu(i["weight"]), stats, dhidden=gpu(i["dhidden"]), rms=rms,
                       channels_first=cf, p=p, seed=seed, call=call, residual=True)
    a = {k: f64(i[k]) for k in ("x", "weight", "bias", "residual")}

    def loss(a):
        s = R.drop(a["x"], p, seed, call) + a["residual"]
        rows = np.moveaxis(s, 1, -1).reshape(-1, 48) if cf else s.reshape(-1, 48)
        o = R.norm_of(rows, a["weight"], a["bias"], 1e-5, rms)[0]
        return (o * rows_of(i["dout"], cf)).sum() + (s * f64(i["dhidden"])).sum()

    rng = np.random.default_rng(3)
    for name, grad in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("residual", "dresidual")):
        v, h = rng.standard_normal(a[name].shape), 1e-5
        d = (loss(dict(a, **{name: a[name] + h * v})) - loss(dict(a, **{name: a[name] - h * v}))) / (2 * h)
        got = f64(g[grad])
        assert abs((got * v).sum() - d) <= 1e-5 * (np.abs(got * v).sum() + 1), name


def test_autograd_and_the_stream_of_blocks():
    """hidden goes from block to block; its gradient is added on the way back."""
    g = torch.Generator().manual_seed(9)
    x, y = (torch.randn(4, 30, 72, generator=g).to(DEV, BF16).requires_grad_(True) for _ in range(2))
    stream = torch.randn(4, 30, 72, generator=g).to(DEV).requires_grad_(True)
    w = (1 + 0.1 * torch.randn(2, 72, generator=g)).to(DEV).requires_grad_(True)
    a, h1 = layer_norm(x, w[0], None, stream, p=0.2, seed=4, call=0)
    b, h2 = layer_norm(y, w[1], None, h1, rms=True, p=0.2, seed=4, call=1)
    (a.float().square().sum() + b.float().sin().sum() + h2.sum()).backward()
    # the same by the plain calls
    with torch.no_grad():
        a1, h1, s1 = layer_norm_fwd(x, w[0].contiguous(), None, stream, p=0.2, seed=4, call=0)
        b1, h2, s2 = layer_norm_fwd(y, w[1].contiguous(), None, h1, rms=True, p=0.2, seed=4, call=1)
        # (torch's own gradients of the losses, in the outputs' dtype)
        db, da = b1.float().cos().to(BF16), (2 * a1.float()).to(BF16)
        g2 = layer_norm_bwd(db, h2, w[1].contiguous(), s2, dhidden=torch.ones_like(h2), rms=True, p=0.2, seed=4, call=1,
                            residual=True, bias=False)
        g1 = layer_norm_bwd(da, h1, w[0].contiguous(), s1, dhidden=g2["dresidual"], p=0.2, seed=4, call=0, residual=True,
                            bias=False)
    assert torch.equal(y.grad, g2["dx"]) and torch.equal(x.grad, g1["dx"]) and torch.equal(stream.grad, g1["dresidual"])
    assert torch.equal(w.grad, torch.stack([g1["dweight"], g2["dweight"]]))


@pytest.mark.parametrize("cf", [False, True], ids=["rows", "cols"])
def test_same_bits_again_on_another_stream_and_into_given_buffers(cf):
    shape = (3, 200, 333) if cf else (999, 200)
    i = make(shape, BF16, F32, seed=11, cf=cf)
    d = {k: gpu(v) for k, v in i.items()}
    kw = dict(channels_first=cf, p=0.25, seed=torch.tensor([5], device=DEV), call=2)
    out, hidden, stats = layer_norm_fwd(d["x"], d["weight"], d["bias"], d["residual"], **kw)
    g = layer_norm_bwd(d["dout"], hidden, d["weight"], stats, dhidden=d["dhidden"], residual=True, **kw)
    side = torch.cuda.Stream()
    made = [torch.empty_like(out), torch.empty_like(hidden), torch.empty_like(stats)]
    ws = torch.empty(layer_norm_bwd_workspace_size(d["dout"], hidden_dtype=F32, channels_first=cf), dtype=torch.uint8,
                     device=DEV)
    torch.cuda.synchronize()
    layer_norm_fwd(d["x"], d["weight"], d["bias"], d["residual"], out=made[0], hidden=made[1], stats=made[2], stream=side, **kw)
    g2 = layer_norm_bwd(d["dout"], made[1], d["weight"], made[2], dhidden=d["dhidden"], residual=True, workspace=ws,
                        grads={k: torch.empty_like(v) for k, v in g.items()}, stream=side, **kw)
    side.synchronize()
    for a, b in zip((out, hidden, stats, *g.values()), (*made, *g2.values())):
        assert torch.equal(a, b)
    # the seed as a number gives the same mask
    kw["seed"] = 5
    assert torch.equal(out, layer_norm_fwd(d["x"], d["weight"], d["bias"], d["residual"], **kw)[0])


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("E", [700, 1000, 1100])
def test_given_workspace_of_the_size_that_is_named(rms, E):
    """Over channels in fp32, where the two norms keep different numbers of them between their passes."""
    print("case: workspace of the norm's gradients", rms, E, flush=True)
    g = torch.Generator(device=DEV).manual_seed(E)
    d, h = torch.randn(1, E, 8192, generator=g, device=DEV), torch.randn(1, E, 8192, generator=g, device=DEV)
    w = torch.ones(E, device=DEV)
    stats = layer_norm_fwd(h, w, rms=rms, channels_first=True)[2]
    n = layer_norm_bwd_workspace_size(d, rms=rms, channels_first=True)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=DEV)
    ws[n:] = 77
    got = layer_norm_bwd(d, h, w, stats, rms=rms, channels_first=True, workspace=ws[:n])
    ref = layer_norm_bwd(d, h, w, stats, rms=rms, channels_first=True)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], ref[k]) for k in ("dx", "dweight", "dbias")) and bool((ws[n:] == 77).all())


@pytest.mark.parametrize("cf", [False, True], ids=["rows", "cols"])
def test_more_than_2_31_elements(cf):
    """The last rows lie behind element 2^31."""
    shape = (1, 64, (1 << 25) + 72) if cf else ((1 << 25) + 72, 64)
    print("case: norm of 2^31 elements", cf, flush=True)
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(shape, dtype=BF16, device=DEV).normal_(generator=g)
    w = torch.randn(64, generator=g, device=DEV)
    out, _, stats = layer_norm_fwd(x, w, rms=True, channels_first=cf, p=0.5, seed=8)
    got = layer_norm_bwd(x, x, w, stats, rms=True, channels_first=cf, p=0.5, seed=8, bias=False)
    torch.cuda.synchronize()
    n = 100
    keep, f = R.mask(n * 64, 0.5, 8, 0, first=x.numel() - n * 64) if not cf else (None, 2.0)
    last = x[..., -n:] if cf else x[-n:]
    rows = rows_of(last, cf)
    if cf:  # element (e, t) is number e L + t
        keep = np.stack([R.mask(n, 0.5, 8, 0, first=(e + 1) * shape[2] - n)[0] for e in range(64)], 1)
    s = np.where(keep.reshape(n, 64), rows, 0) * f
    ref, _, m, fac = R.norm_of(s, f64(w), None, 1e-5, True)
    o = rows_of(out[..., -n:] if cf else out[-n:], cf)
    assert (np.abs(o - ref) <= (half(BF16) + 200 * U) * np.abs(ref) + 1e-30).all()
    assert (np.abs(f64(stats[1, -n:]) - fac) <= 100 * U * fac).all()
    ds = R.norm_grads(rows, rows, f64(w), m, f64(stats[1, -n:]), None, True)[0]
    dx = rows_of(got["dx"][..., -n:] if cf else got["dx"][-n:], cf)
    ref = np.where(keep.reshape(n, 64), ds, 0) * f
    scale = f64(stats[1, -n:])[:, None] * 4 * (np.abs(rows * f64(w)) + np.abs(rows) * 5)
    assert (np.abs(dx - ref) <= half(BF16) * np.abs(ref) + 200 * U * scale).all()


def test_gradients_of_2_30_columns():
    """A row of all the elements that a row may have: the join of the sums takes 2^32 threads and more."""
    print("case: norm gradients of 2^30 columns", flush=True)
    E, g = 1 << 30, torch.Generator(device=DEV).manual_seed(6)
    d, h = (torch.empty(1, E, dtype=BF16, device=DEV).normal_(generator=g) for _ in range(2))
    w = torch.ones(E, device=DEV)
    stats = torch.tensor([[0.25], [0.5]], device=DEV)
    got = layer_norm_bwd(d, h, w, stats)
    torch.cuda.synchronize()
    for lo in (0, (1 << 29) - 50, E - 100):
        s = slice(lo, lo + 100)
        dd, hh = f64(d[0, s]), f64(h[0, s])
        want = dd * (hh - 0.25) * 0.5
        assert np.array_equal(f64(got["dbias"][s]), dd)
        # a difference, a product with 1/2 (exact), a product
        assert (np.abs(f64(got["dweight"][s]) - want) <= 3 * U * (np.abs(dd) * (np.abs(hh) + 0.25))).all()
