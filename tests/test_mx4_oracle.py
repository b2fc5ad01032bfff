"""Pins for the MXFP4 oracle and for the layout of given choices: E2M1 by enumeration of its bit
fields, the shared exponent by repeated doubling, worked blocks, the cases without a value."""
import itertools

import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import mx4_oracle as M4


def _fields():
    """E2M1's magnitudes from sign-exponent-mantissa (bias 1, exponent 0 subnormal)."""
    return [(m / 2.0 if e == 0 else (1 + m / 2.0) * 2.0 ** (e - 1)) for e, m in itertools.product(range(4), range(2))]


def test_values_are_the_bit_fields():
    assert list(M4.VALUES) == _fields()
    assert M4.e2m1_decode(np.arange(16)).tolist() == _fields() + [-v for v in _fields()]


def test_encode_takes_the_nearest_ties_to_even():
    v = _fields()
    ys = np.concatenate([np.linspace(-9, 9, 14401), np.array(v), -np.array(v)])
    for y in ys:
        a = abs(y)
        best = min(range(8), key=lambda c: (abs(min(a, 6.0) - v[c]), c % 2))
        assert int(M4.e2m1_encode(y)) == (best | (8 if np.signbit(y) else 0)), y


@pytest.mark.parametrize("amax,code", [(6.0, 127), (4.0, 127), (3.999, 126), (1.0, 125), (8.0, 128), (2.0 ** -125, 0),
                                       (2.0 ** -140, 0), (2.0 ** 127, 252), (0.0, 0), (np.inf, 255), (np.nan, 255)])
def test_scale_code(amax, code):
    x = np.zeros(64)
    x[40] = -amax
    x[3] = 1.0
    c, s, v = M4.quantize(x)
    assert s.tolist() == [125, code]
    if code in (0, 255):
        assert (c[32:] == 0).all() or amax > 0 and code == 0
    if code == 255:
        assert np.isnan(v[32:]).all() and np.isfinite(v[:32]).all()


def test_worked_block():
    x = np.zeros(32)
    x[:8] = [5.0, -5.1, 2.5, 3.5, 0.25, -0.25, 0.26, 7.9]
    c, s, v = M4.quantize(x)
    assert s.tolist() == [127]
    assert v[:8].tolist() == [4.0, -6.0, 2.0, 4.0, 0.0, -0.0, 0.5, 6.0]
    assert np.array_equal(M4.dequantize(M4.pack(c), s), v)
    assert M4.pack(np.array([1, 2, 15, 0], dtype=np.uint8)).tolist() == [0x21, 0x0F]


def test_layout_is_the_routed_layout_where_nothing_is_dropped():
    rng = np.random.default_rng(0)
    idx = np.stack([np.stack([rng.permutation(16)[:4] for _ in range(37)]) for _ in range(2)]).astype(np.int32)
    e2l = np.full(16, -1, dtype=np.int32)
    e2l[[3, 5, 0, 15]] = [2, 0, 1, 3]
    a, b = M4.layout(idx, e2l, 4), O.layout(idx, e2l, 4)
    for n in ("counts", "offsets", "slot_of"):
        assert np.array_equal(a[n], b[n]), n
    assert np.array_equal(a["pull_src"], b["pull_src"][: len(a["pull_src"])])


def test_layout_drops():
    idx = np.array([[[0, -1], [1, 0], [-1, -1], [-1, 1]]], dtype=np.int32)
    a = M4.layout(idx, np.array([1, 0], dtype=np.int32), 2)
    assert a["counts"].tolist() == [2, 2] and a["offsets"].tolist() == [0, 2, 4]
    assert a["slot_of"].tolist() == [[[2, -1], [0, 3], [-1, -1], [-1, 1]]]
    assert a["pull_src"].tolist() == [[0, 1], [0, 3], [0, 0], [0, 1]]
    y = M4.merge(np.array([[1.0], [2.0], [4.0], [8.0]]), a["slot_of"], np.full((1, 4, 2), 0.5))
    assert y[0, :, 0].tolist() == [2.0, 4.5, 0.0, 1.0]
