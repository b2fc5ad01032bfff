"""Pins of the oracle of the norm, the grouped products and the AdamW step: closed forms, and gradients against differences."""
import numpy as np
import pytest

from oracle import more_oracle as M
from oracle import mx_oracle as M8


@pytest.mark.parametrize("d,residual", [(1, False), (7, True), (64, True)])
def test_norm_gradients_against_differences(d, residual):
    r = np.random.default_rng(d)
    h, dy, gamma = r.standard_normal((3, d)), r.standard_normal((3, d)), r.standard_normal(d)
    dh = r.standard_normal((3, d)) if residual else None

    def loss(h, gamma):
        s, n, _ = M.norm(h, None, gamma, 1e-3)
        return (n * dy).sum() + ((s * dh).sum() if residual else 0.0)

    dx, dgamma, _, _ = M.norm_backward(dy, h, gamma, dh, 1e-3)
    step = 1e-5                                   # central differences: error of the order of step^2 and 1e-16 / step
    for i in range(3):
        for j in range(d):
            e = np.zeros_like(h)
            e[i, j] = step
            assert abs((loss(h + e, gamma) - loss(h - e, gamma)) / (2 * step) - dx[i, j]) < 1e-7 * (1 + abs(dx).max())
    for j in range(d):
        e = np.zeros(d)
        e[j] = step
        assert abs((loss(h, gamma + e) - loss(h, gamma - e)) / (2 * step) - dgamma[j]) < 1e-7 * (1 + abs(dgamma).max())


def test_norm_of_equal_values():
    s, n, rstd = M.norm(np.full((2, 5), 3.0), np.full((2, 5), 1.0), np.arange(5.0), 0.0)
    assert (s == 4).all() and np.allclose(rstd, 0.25) and np.allclose(n, np.arange(5.0))


@pytest.mark.parametrize("layout", [0, 1])
def test_product_gradients_against_differences(layout):
    r = np.random.default_rng(layout)
    off = [0, 2, 2, 7]
    x, dy = r.standard_normal((8, 3)), r.standard_normal((8, 4))
    w = r.standard_normal((3, 4, 3) if layout == 0 else (3, 3, 4))
    loss = lambda x, w: np.nansum(M.grouped(x, w, off, layout)[0] * dy)          # noqa: E731
    dx, _ = M.grouped(dy, w, off, 1 - layout)
    dw, _ = M.grouped_wgrad(x, dy, off, layout)
    assert (dw[1] == 0).all() and np.isnan(dx[7]).all()
    for t, grad in ((x, dx), (w, dw)):
        for i in np.ndindex(t.shape):
            if np.isnan(grad[i]):
                continue
            keep = t[i]
            t[i] = keep + 1.0
            up = loss(x, w)
            t[i] = keep
            assert abs(up - loss(x, w) - grad[i]) < 1e-12 * 100      # linear: the difference is the gradient


def test_state_codes_nearest_equal_the_codec_where_nothing_saturates():
    r = np.random.default_rng(3)
    v = (r.standard_normal(128 * 64) * np.exp(r.standard_normal(128 * 64) * 4)).astype(np.float32)
    codes, scales = M.state_codes(v, None, False)
    rc, rs, rv = M8.quantize(v.astype(np.float64).reshape(-1, 128))[:3]
    b = np.abs(v.reshape(-1, 32)).max(-1)
    within = b <= 448 * np.exp2(np.floor(np.log2(b)) - 8)
    assert within.any() and not within.all()
    rc = np.where(np.asarray(rc) == 128, 0, rc)              # a state that rounds to zero has no sign
    assert np.array_equal(codes.reshape(-1, 32)[within], rc.reshape(-1, 32)[within])
    assert np.array_equal(scales[within], np.asarray(rs).reshape(-1)[within])
    # where it would, the scale is one larger and the block's maximum within half a step of itself
    val = M.state_values(codes, scales).reshape(-1, 32)
    assert (np.abs(np.abs(val).max(-1) - b) <= b / 16 + 1e-300).all()


def test_state_codes_are_unbiased_and_neighbours():
    r = np.random.default_rng(4)
    v = np.tile((r.standard_normal(128) * np.exp(r.standard_normal(128) * 3)).astype(np.float32), 512)
    bits = M.random_bits(99, 7, 3, v.size, 0)
    codes, scales = M.state_codes(v, bits & np.uint64(0xFFFF), False)
    val = M.state_values(codes, scales).reshape(512, 128)
    unit = np.exp2(scales.reshape(512, 4).astype(np.float64) - 127)[0].repeat(32)
    step = np.maximum(np.exp2(np.floor(np.log2(np.abs(v[:128]) / unit)) - 3), 2.0 ** -9) * unit
    assert (np.abs(val - v[:128]) < step).all()
    # 512 draws of a step's indicator: the mean is off by 5 of its deviations at most (one in 1.7 million; 128 values)
    assert (np.abs(val.mean(0) - v[:128]) <= 5 * step * 0.5 / np.sqrt(512) + 2.0 ** -16 * step).all()
    roots, sc = M.state_codes(np.abs(v), (bits >> np.uint64(16)), True)
    assert (M.state_values(roots, sc)[np.abs(v) > 0] > 0).all()


def test_random_bits_are_spread():
    """Bytes of many places, steps, tensors and seeds: every value about as often (chi-squared of 255 degrees of freedom,
    mean 255, deviation 22.6: below 255 + 6 * 22.6), and neighbours without correlation."""
    draws = [M.random_bits(1, 1, 0, 1 << 16, 0), M.random_bits(1, 1, 0, 1 << 16, 1),
             np.array([M.random_bits(1, s, 0, 1, 0)[0] for s in range(4096)]),
             np.array([M.random_bits(s, 1, 0, 1, 0)[0] for s in range(4096)]),
             np.array([M.random_bits(1, 1, s, 1, 0)[0] for s in range(4096)])]
    for z in draws:
        for shift in (0, 8, 16, 24):
            n = np.bincount(((z >> np.uint64(shift)) & np.uint64(255)).astype(int), minlength=256)
            assert ((n - z.size / 256) ** 2 / (z.size / 256)).sum() < 255 + 6 * 22.6
        f = z.astype(np.float64) / 2 ** 32 - 0.5
        assert abs((f[1:] * f[:-1]).mean() * 12) < 6 / np.sqrt(z.size)
    a, b = (d.astype(np.float64) / 2 ** 32 - 0.5 for d in draws[:2])
    assert abs((a * b).mean() * 12) < 6 / np.sqrt(a.size)


def test_adamw_first_step_moves_by_the_rate():
    """From zero states the first step moves every value by lr, whatever its gradient's size."""
    g = np.array([1e-3, -5.0, 2.0], np.float32)
    m, v = M.moments(np.zeros(3), np.zeros(3), g, 0.9, 0.999)
    p, away = M.adamw(np.ones(3), m, v, 0.01, 0.9, 0.999, 1e-12, 1, 0.1)
    assert np.allclose(p, 1 * (1 - 0.001) - 0.01 * np.sign(g), rtol=1e-6)
    assert np.allclose(away * np.sign(g), 0.01 * np.sign(g), rtol=1e-6)
