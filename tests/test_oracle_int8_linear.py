"""Pins of the int8 linear oracle (oracle/int8_linear.py), CPU only: hand-made codes with ties,
fractions, and gradients against differences of the layer that the codes stand for."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8_linear as il


def test_codes_by_hand():
    x = np.float32([[127, 63.5, 62.5, -63.5, 1.5, 0.5, 0.49, 0], [2, 1, -1, 0.25, 0, 0, 0, 0], [0] * 8,
                    [1, np.inf, 0, 0, 0, 0, 0, 0], [1, np.nan, 0, 0, 0, 0, 0, 0]])
    codes, scales = il.quant_rows(x)
    assert codes[0].tolist() == [127, 64, 62, -64, 2, 0, 0, 0]          # halves go to even
    assert codes[1].tolist() == [127, 64, -64, 16, 0, 0, 0, 0]          # absmax / 2 is a tie at 63.5
    assert not codes[2:].any() and scales[2] == 1 and np.isnan(scales[3:]).all()
    assert scales[0] == 1 and scales[1] == np.float32(2) / np.float32(127)


@pytest.mark.parametrize("power", [0, -120, 100])
def test_codes_against_fractions(power):
    x = (np.random.default_rng(3).standard_normal((6, 40)) * 2.0 ** power).astype(np.float32)
    codes, _ = il.quant_rows(x)
    for row, got in zip(x, codes):
        top = max(abs(Fraction(float(a))) for a in row)
        assert got.tolist() == [round(Fraction(float(a)) * 127 / top) for a in row]    # round() is half to even


def test_layer_and_gradients():
    rng = np.random.default_rng(5)
    codes, scales = il.quant_rows(rng.standard_normal((5, 16)))
    wc, ws = il.quant_rows(rng.standard_normal((8, 16)))
    bias, dy = rng.standard_normal(8), rng.standard_normal((5, 8))
    y, _ = il.linear(codes, scales, wc, ws, bias)
    np.testing.assert_allclose(y, il.values(codes, scales) @ il.values(wc, ws).T + bias, rtol=1e-13)
    x, w, e = il.values(codes, scales), il.values(wc, ws), 1e-4
    dw, dx = il.grad_weight(dy, codes, scales)[0], il.grad_input(dy, wc, ws)[0]
    loss = lambda a, b: float(((a @ b.T + bias) * dy).sum())               # noqa: E731
    for at in [(0, 0), (3, 7), (7, 15)]:
        d = np.zeros_like(w)
        d[at] = e
        assert dw[at] == pytest.approx((loss(x, w + d) - loss(x, w - d)) / (2 * e), abs=1e-8)
    for at in [(0, 0), (4, 15)]:
        d = np.zeros_like(x)
        d[at] = e
        assert dx[at] == pytest.approx((loss(x + d, w) - loss(x - d, w)) / (2 * e), abs=1e-8)
