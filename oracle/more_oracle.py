"""CPU oracle for the operators before, beside and behind the layer: the RMS norm with the residual's addition and its
gradients, products grouped by expert and theirs, and the AdamW step with states in 32 or 8 bits.

TEST INFRASTRUCTURE ONLY (imported by tests/ only; shares no code with the HIP path).  Formulas in 64 bits; the AdamW
step's states are computed in float32 in the order that the header states, so that their bits can be compared.
"""
from __future__ import annotations

import numpy as np

from . import mx_oracle as M8


# ------------------------------------------------------------------------------------------------ norm
def norm(x, residual, gamma, eps):
    """(sum, n, rstd) of rows in 64 bits."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    g = 1.0 if gamma is None else np.asarray(gamma, np.float64)
    return s, s * rstd * g, rstd


def norm_backward(dy, h, gamma, dh, eps):
    """(dx, dgamma, bound of dx's terms, bound of dgamma's): the bounds are the sums of magnitudes."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    g = np.ones(h.shape[1]) if gamma is None else np.asarray(gamma, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    u = dy * g
    dot, mag = (u * h).mean(-1, keepdims=True), np.abs(u * h).mean(-1, keepdims=True)
    dx = rstd * (u - h * rstd ** 2 * dot)
    bound = rstd * (np.abs(u) + np.abs(h) * rstd ** 2 * mag)
    if dh is not None:
        dx = dx + dh
        bound = bound + np.abs(dh)
    return dx, (dy * h * rstd).sum(0), bound, np.abs(dy * h * rstd).sum(0)


# ------------------------------------------------------------------------------------------------ products
def grouped(x, w, offsets, layout):
    """(y, sum of the magnitudes of its terms); rows of no group are NaN."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    n = w.shape[1] if layout == 0 else w.shape[2]
    y, mag = np.full((x.shape[0], n), np.nan), np.full((x.shape[0], n), np.nan)
    for g, (a, b) in enumerate(zip(offsets, offsets[1:])):
        m = w[g].T if layout == 0 else w[g]
        y[a:b], mag[a:b] = x[a:b] @ m, np.abs(x[a:b]) @ np.abs(m)
    return y, mag


def grouped_wgrad(x, dy, offsets, layout):
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    a, b = (dy, x) if layout == 0 else (x, dy)
    parts = [(a[i:j].T @ b[i:j], np.abs(a[i:j]).T @ np.abs(b[i:j])) for i, j in zip(offsets, offsets[1:])]
    return np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])


# ------------------------------------------------------------------------------------------------ AdamW
def mix(z):
    """The header's mixing of 32 bits, on uint64 arrays that hold 32."""
    z = np.asarray(z, np.uint64) & np.uint64(0xFFFFFFFF)
    for shift, odd in ((16, 0x9E3779B9), (15, 0xBB67AE85)):
        z = z ^ (z >> np.uint64(shift))
        z = (z * np.uint64(odd)) & np.uint64(0xFFFFFFFF)
    return z ^ (z >> np.uint64(16))


def random_bits(seed, step, tensor, n, which, first=0):
    """32 bits a value of one tensor; which = 0 for the states, 1 for a bf16 param without a master."""
    i = np.arange(first, first + n, dtype=np.uint64)
    key = mix(mix(mix(mix(seed & 0xFFFFFFFF) + np.uint64(seed >> 32)) + np.uint64(step & 0xFFFFFFFF)) + np.uint64(tensor))
    key = mix(mix(key + (i >> np.uint64(32))) + np.uint64(1 + which))
    return mix((i & np.uint64(0xFFFFFFFF)) + key)


def state_codes(v, r16, root):
    """(E4M3 codes, scale codes) of float32 states, a multiple of 128 of them; r16: 16 random bits a value, None for
    nearest even."""
    v = np.asarray(v, np.float32)
    b = v.reshape(-1, 32).astype(np.float64)
    wild = ~np.isfinite(b).all(-1)
    top = np.where(wild, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    e = np.frexp(top)[1] - 9
    e = np.clip(e + (top > np.ldexp(448.0, e)), -127, 127)
    y = np.where(wild[:, None], 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)) / np.ldexp(1.0, e)[:, None])
    step = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)
    if r16 is None:
        q = np.rint(y / step)
    else:
        part = np.asarray(r16, np.float64).reshape(-1, 32) / 65536
        # below E4M3's smallest power of two the 20 bits that are cut off are themselves cut from more
        units = np.where(y < 2.0 ** -6, np.floor(y * 2.0 ** 29) / 2.0 ** 20, y / step)
        q = np.floor(units + part)
    q = np.minimum(q * step, 448.0)
    if root:
        q = np.where((b > 0) & (q == 0), 2.0 ** -9, q)
    codes = M8.e4m3_encode(q).astype(np.int64) | np.where((q > 0) & np.signbit(b) & (not root), 128, 0)
    blank = (wild | (top == 0))[:, None]
    return np.where(blank, 0, codes).astype(np.uint8).reshape(v.shape), \
        np.where(wild, 255, np.where(top > 0, e + 127, 0)).astype(np.uint8)


def state_values(codes, scales):
    c = np.asarray(codes).astype(np.int64)
    field, part = (c >> 3) & 15, (c & 7) / 8
    size = np.where(field > 0, (1 + part) * np.exp2(field - 7.0), part * 2.0 ** -6)
    unit = np.where(np.asarray(scales) == 255, np.nan, np.exp2(np.asarray(scales, np.float64) - 127))
    return (np.where(c & 128, -size, size).reshape(-1, 32) * unit[:, None]).reshape(c.shape)


def moments(m, v, g, beta1, beta2):
    """Both states after a gradient, in float32, each operation rounded once."""
    f = np.float32
    m, v, g = (np.asarray(t, f) for t in (m, v, g))
    with np.errstate(all="ignore"):
        m = f(beta1) * m + f(1 - beta1) * g
        v = f(beta2) * v + (f(1 - beta2) * g) * g
    return m, v


def adamw(p, m, v, lr, beta1, beta2, eps, step, wd):
    """(the param after the step in 64 bits, the magnitude of its change) from the states that the step has made."""
    p, m, v = (np.asarray(t, np.float64) for t in (p, m, v))
    away = lr * (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * wd) - away, np.abs(away)
