"""Plain 64-bit forms of the training operators (numpy / torch on the CPU), for the tests."""
from __future__ import annotations

import numpy as np
import torch


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def conv_grads(x, w, b, init, dout, dfinal):
    """The conv's gradients from the definition.  Arrays as conv1d_fwd's; returns dx, dweight, dbias, dinit."""
    B, D, L = x.shape
    H = w.shape[1] - 1
    xs = np.zeros((B, D, H + L))
    xs[..., H:] = x
    if init is not None:
        xs[..., :H] = init
    a = np.zeros((B, D, L)) + (0.0 if b is None else b[None, :, None])
    for k in range(H + 1):
        a += w[None, :, k:k + 1] * xs[..., k:k + L]
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-a))
    g = dout * s * (1 + a * (1 - s))
    dxs = np.zeros_like(xs)
    dw = np.zeros_like(w)
    for k in range(H + 1):
        dxs[..., k:k + L] += w[None, :, k:k + 1] * g
        dw[:, k] = (g * xs[..., k:k + L]).sum((0, 2))
    if dfinal is not None and H:
        dxs[..., L:] += dfinal
    return dxs[..., H:], dw, g.sum((0, 2)), dxs[..., :H]


def embed_grad(tokens, rows, V, scale):
    """(dweight, its sums of magnitudes, occurrences per token); rows: [T, E]."""
    t = np.asarray(tokens).reshape(-1)
    ok = (t >= 0) & (t < V)
    dw, mag, n = np.zeros((V, rows.shape[1])), np.zeros((V, rows.shape[1])), np.zeros(V)
    np.add.at(dw, t[ok], rows[ok])
    np.add.at(mag, t[ok], np.abs(rows[ok]))
    np.add.at(n, t[ok], 1)
    return dw * scale, mag * abs(scale), n


M32 = 0xFFFFFFFF


def mix(x):
    x = np.asarray(x, np.uint64)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x6A09E667)) & np.uint64(M32)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xBB67AE85)) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def random_bits(seed, step, tensor, n):
    """The 32-bit random numbers of a tensor's elements."""
    key = mix(seed & M32)
    if seed >> 32:
        key = mix((key + np.uint64(seed >> 32)) & np.uint64(M32))
    key = mix((key + np.uint64(step)) & np.uint64(M32))
    key = mix((key + np.uint64(tensor)) & np.uint64(M32))
    i = np.arange(n, dtype=np.uint64)
    return mix((i * np.uint64(0x9E3779B9) + key) & np.uint64(M32))


def blocks(a):
    """a, padded with zeros to whole blocks of 128, as [blocks, 128]."""
    return np.concatenate([a, np.zeros(-len(a) % 128, a.dtype)]).reshape(-1, 128)


def decode(code, base, signed):
    """The numbers that 8-bit codes stand for (fp32)."""
    c = code.astype(np.int64)
    mag = c & 127 if signed else c
    bits = np.where(mag > 0, (blocks(mag) + base.astype(np.int64)[:, None]).reshape(-1)[:len(c)] << 20, 0)
    v = bits.astype(np.uint32).view(np.float32)
    return np.where(c >= 128, -v, v) if signed else v


def encode(x, r, signed):
    """(codes, bases) of fp32 x: bit for bit what include/ssm_scan.h describes."""
    top = 127 if signed else 255
    a = np.abs(x).view(np.uint32).astype(np.int64)
    base = np.maximum(((blocks(a).max(1) + 0xFFFFF) >> 20) - top, 0)
    K = np.repeat(base, 128)[:len(x)]
    q = ((a + (r.astype(np.int64) << 4) + 8) >> 20) - K
    if signed:
        least = ((K + 1) << 20).astype(np.uint32)
        u = (r.astype(np.float64) + 0.5) / 65536
        under = np.abs(x).astype(np.float64) > least.view(np.float32).astype(np.float64) * u
        q = np.where(a < least, under, np.clip(q, 0, top)) + np.where(x < 0, 128, 0)
    else:
        q = np.where(a > 0, np.clip(q, 1, top), 0)
    return q.astype(np.uint8), base.astype(np.int16)


def moments32(m, v, g, b1, b2):
    """The moments in fp32, every product and sum rounded once, in the order of the definition."""
    f = np.float32
    m1 = m.astype(f) * f(b1) + g.astype(f) * f(1 - b1)
    v1 = v.astype(f) * f(b2) + g.astype(f) * f(1 - b2) * g.astype(f)
    return m1.astype(f), v1.astype(f)


def adamw64(p, m, v, lr, b1, b2, eps, wd, step):
    """(p, update) of one step in 64 bits, from the step's moments.  These are fp32 numbers and rounded: where
    b1 m and (1 - b1) g cancel, their rounding is more than any of an update's own."""
    u = lr * (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * wd) - u, u
