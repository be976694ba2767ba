"""Plain 64-bit forms of the residual block's operators (numpy on the CPU), for the tests."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def philox(counter, key):
    """Philox4x32 with ten rounds, on Python integers: four words from four and two."""
    c, k, m = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def mask(n, p, seed, call, first=0):
    """(kept, factor) of elements first .. first + n - 1."""
    m = np.uint64(0xFFFFFFFF)
    j = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    c = [j & m, j >> np.uint64(32), np.full_like(j, call & 0xFFFFFFFF), np.full_like(j, call >> 32 & 0xFFFFFFFF)]
    k = [np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32 & 0xFFFFFFFF)]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ k[0], b & m, (a >> np.uint64(32)) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + np.uint64(0x9E3779B9)) & m, (k[1] + np.uint64(0xBB67AE85)) & m]
    half = np.stack([h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1).reshape(-1)
    T = int(np.rint(p * 65536))
    return half[first % 8:][:n] >= T, 65536 / (65536 - T) if T < 65536 else 0.0


def drop(x, p, seed, call):
    keep, f = mask(x.size, p, seed, call)
    return np.where(keep.reshape(x.shape), x, 0.0) * f


def norm(x, w, b, residual, eps, rms, p=0.0, seed=0, call=0):
    """x: [rows, E] (in the tensor's memory order).  (out, hidden, mean, factor)."""
    s = x if p == 0.0 else drop(x, p, seed, call)
    s = s if residual is None else s + residual
    return (*norm_of(s, w, b, eps, rms), )


def norm_of(s, w, b, eps, rms):
    m = np.zeros(s.shape[0]) if rms else s.mean(1)
    d = s - m[:, None]
    f = 1 / np.sqrt((d * d).mean(1) + eps)
    out = d * f[:, None] * (1.0 if w is None else w) + (0.0 if b is None else b)
    return out, s, m, f


def norm_grads(dout, s, w, m, f, dhidden, rms):
    """(ds, dweight, dbias); s, dout: [rows, E]."""
    xh = (s - m[:, None]) * f[:, None]
    g = dout * (1.0 if w is None else w)
    ds = g - xh * (g * xh).mean(1, keepdims=True)
    if not rms:
        ds = ds - g.mean(1, keepdims=True)
    ds = ds * f[:, None]
    return ds + (0.0 if dhidden is None else dhidden), (dout * xh).sum(0), dout.sum(0)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def _col(v):
    return 0.0 if v is None else v[None, :, None]


def gates(r, i, decay, rb, ib):
    sr, si = sigmoid(r + _col(rb)), sigmoid(i + _col(ib))
    la = -decay[None, :, None] * sr
    return sr, si, np.exp(la), -np.expm1(2 * la)


def recurrence(x, r, i, decay, rb=None, ib=None, z=None, init=None, reverse=False):
    """(out, last, states [B,D,L+1] in the order of the steps, bound on their fp32 error), step by step."""
    sr, si, a, w = gates(r, i, decay, rb, ib)
    v = np.sqrt(w) * si * x
    # fp32 errors, relative: of the gates (the exponential's argument, itself, the sum, the reciprocal), of a = e^-t/2, of
    # w = 1 - a^2 (a series below t = 1/4), of v
    # (an argument past 200 gives 0 or 1 to the last bit of fp32, infinite ones too)
    er, ei = ((2 * np.minimum(np.abs(q), 200) + 5) * U for q in (r + _col(rb), i + _col(ib)))
    t = 2 * decay[None, :, None] * sr
    ea = t / 2 * (er + 2 * U) + 2 * U
    ew = np.where(t < 0.25, er + 12 * U, 2 * (1 - w) / np.maximum(w, 0.2) * ea + 5 * U)
    ev = ew / 2 + ei + 4 * U
    if reverse:
        a, v, ea, ev = (q[..., ::-1] for q in (a, v, ea, ev))
    B, D, L = x.shape
    h = np.zeros((B, D, L + 1))
    if init is not None:
        h[..., 0] = init
    mag, err = np.abs(h), np.zeros_like(h)
    for k in range(L):
        h[..., k + 1] = a[..., k] * h[..., k] + v[..., k]
        mag[..., k + 1] = a[..., k] * mag[..., k] + np.abs(v[..., k])
        err[..., k + 1] = a[..., k] * (err[..., k] + mag[..., k] * (ea[..., k] + 2 * U)) + np.abs(v[..., k]) * (ev[..., k] + U)
    # the maps of lanes and waves are composed in a tree: a lane's 8 steps, 12 and 4 more, each a product and a sum
    err += 48 * U * mag
    out, bound = h[..., 1:], err[..., 1:]
    if reverse:
        out, bound = out[..., ::-1], bound[..., ::-1]
    if z is not None:
        f = z * sigmoid(z)
        bound = bound * np.abs(f) + np.abs(out * f) * (2 * np.abs(z) + 6) * U
        out = out * f
    return out, h[..., -1], h, bound, err


def recurrence_grads(x, r, i, decay, rb, ib, z, init, dout, dlast, reverse=False):
    """dict of gradients, from the formulas step by step."""
    sr, si, a, w = gates(r, i, decay, rb, ib)
    q = np.sqrt(w)
    _, _, h, _, _ = recurrence(x, r, i, decay, rb, ib, z, init, reverse)
    turn = (lambda t: t[..., ::-1]) if reverse else (lambda t: t)
    before, after = turn(h[..., :-1]), turn(h[..., 1:])
    g, dz = dout, None
    if z is not None:
        s = sigmoid(z)
        dz = dout * after * s * (1 + z * (1 - s))
        g = dout * z * s
    ta, tg = turn(a), turn(g)
    F = np.zeros(x.shape[:2]) if dlast is None else dlast
    G = np.zeros_like(x)
    for k in range(x.shape[2] - 1, -1, -1):
        G[..., k] = tg[..., k] + F
        F = ta[..., k] * G[..., k]
    G = turn(G)
    iq = 1 / np.maximum(q, 2.0 ** -50)
    dla = G * (a * before - si * x * a * a * iq)
    dr = -decay[None, :, None] * dla * sr * (1 - sr)
    di = G * q * x * si * (1 - si)
    return dict(dx=G * q * si, dr=dr, di=di, dz=dz, ddecay=-(dla * sr).sum((0, 2)), dr_bias=dr.sum((0, 2)),
                di_bias=di.sum((0, 2)), dinitial_state=F)


def checkpoint_steps(B, D, L, v, blocks, reverse=False):
    """The number of steps before each checkpoint [B, D, blocks]; v: elements in 16 bytes."""
    row = np.arange(B * D).reshape(B, D, 1)
    m = -(row + 1) * L % v if reverse else row * L % v
    return np.clip(np.arange(blocks) * 64 * v - m, 0, L)
