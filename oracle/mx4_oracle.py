"""CPU oracle for the MXFP4 forward: E2M1 elements with one E8M0 scale per 32 along K, and for the
layer under given choices and gate weights.

TEST INFRASTRUCTURE ONLY (imported by tests/ only; shares no code with the HIP path).

The format is OCP Microscaling (MX) v1.0 MXFP4: E2M1 (bias 1, one mantissa bit, the subnormal
0.5, largest value 6, no NaN or infinity), scale exponent floor(log2 amax) - 2 clamped to
[-127, 127], elements rounded to nearest with ties to the even code and saturated to +-6.  An
all-zero block has scale code 0 and zero codes; a block with a NaN or an infinity has scale code
255 and zero codes.
"""
from __future__ import annotations

import numpy as np

from . import moe_oracle as O

BLOCK = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_encode(y: np.ndarray) -> np.ndarray:
    """Code (0..15, sign in bit 3) of the nearest E2M1 value of y, ties to the even code."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(y), 6.0)
    hi = np.searchsorted(VALUES, a, side="left")           # VALUES[hi] >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - VALUES[lo], VALUES[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (a == VALUES[hi])
    return (np.where(up, hi, lo) | (np.signbit(y).astype(np.int64) << 3)).astype(np.uint8)


def e2m1_decode(code: np.ndarray) -> np.ndarray:
    c = np.asarray(code, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * VALUES[c & 7]


def scale_value(code: np.ndarray) -> np.ndarray:
    c = np.asarray(code, dtype=np.float64)
    return np.where(c == 255, np.nan, np.exp2(c - 127.0))


def quantize(x: np.ndarray):
    """(codes 0..15 uint8 [..., K], scale codes uint8 [..., K/32], values float64 [..., K])."""
    x = np.asarray(x, dtype=np.float64)
    xb = x.reshape(*x.shape[:-1], -1, BLOCK)
    wild = ~np.isfinite(xb).all(-1)
    amax = np.where(wild, 1.0, np.abs(np.where(np.isfinite(xb), xb, 0.0)).max(-1))
    _, ex = np.frexp(amax)
    e = np.clip(ex - 1 - 2, -127, 127)
    sc = np.where(wild, 255, np.where(amax > 0, e + 127, 0)).astype(np.uint8)
    blank = (wild | (amax == 0))[..., None]
    codes = np.where(blank, 0, e2m1_encode(np.where(blank, 0.0, xb) / np.exp2(e.astype(np.float64))[..., None])).astype(np.uint8)
    val = e2m1_decode(codes) * scale_value(sc)[..., None]
    return codes.reshape(x.shape), sc, val.reshape(x.shape)


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed: np.ndarray) -> np.ndarray:
    return np.stack((packed & 15, packed >> 4), axis=-1).reshape(*packed.shape[:-1], -1)


def dequantize(packed: np.ndarray, scale_codes: np.ndarray) -> np.ndarray:
    """Values of packed codes [..., K/2] with row-major scale codes [..., K/32]."""
    v = e2m1_decode(unpack(packed))
    return v * np.repeat(scale_value(scale_codes), BLOCK, axis=-1)


# ------------------------------------------------------------------- given choices
def layout(idx: np.ndarray, expert_to_local: np.ndarray, E_local: int) -> dict:
    """Counts, offsets, pull schedule and slots of choices [R][T][k] in which -1 is no expert, by
    plain loops in (r, t, j) order."""
    R, T, k = idx.shape
    counts = np.zeros(len(expert_to_local), dtype=np.int32)
    lists = [[] for _ in range(E_local)]
    for r in range(R):
        for t in range(T):
            for j in range(k):
                e = int(idx[r, t, j])
                if e < 0:
                    continue
                counts[e] += 1
                l = int(expert_to_local[e])
                if l >= 0:
                    lists[l].append((r, t, j))
    offsets = np.zeros(E_local + 1, dtype=np.int32)
    offsets[1:] = np.cumsum([len(v) for v in lists])
    slot_of = np.full(idx.shape, -1, dtype=np.int32)
    pull = np.zeros((int(offsets[-1]), 2), dtype=np.int32)
    s = 0
    for v in lists:
        for (r, t, j) in v:
            slot_of[r, t, j] = s
            pull[s] = (r, t)
            s += 1
    return {"counts": counts, "offsets": offsets, "slot_of": slot_of, "pull_src": pull}


def merge(rows: np.ndarray, slot_of: np.ndarray, w) -> np.ndarray:
    """y[r][t] = sum_j w rows[slot] (w None: 1)."""
    y = np.zeros((*slot_of.shape[:2], rows.shape[1]))
    for j in range(slot_of.shape[2]):
        s = slot_of[:, :, j]
        v = np.asarray(rows, dtype=np.float64)[np.maximum(s, 0)] if rows.shape[0] else np.zeros_like(y)
        g = 1.0 if w is None else np.asarray(w, dtype=np.float64)[:, :, j, None]
        y += np.where((s >= 0)[..., None], v * np.where((s >= 0)[..., None], g, 0.0), 0.0)
    return y


def ffn_q(rows: np.ndarray, w1, w3, w2):
    """One expert on quantised values: h quantised along F.  Returns (ye, h before rounding)."""
    a, b = rows @ w1.T, rows @ w3.T
    h = O.silu(a) * b
    return quantize(h)[2] @ w2.T, h
