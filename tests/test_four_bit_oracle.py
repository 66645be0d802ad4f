"""Pins of the four-bit oracle (oracle/four_bit.py): hand-worked values, torch's own decoders, central differences of its
forward formulas for the gradients."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
import oracle.four_bit as F
import workloads as W


@pytest.mark.parametrize("amax, code", [(6.0, 127), (6.0001, 128), (3.0, 126), (1.0, 125), (0.75, 124), (0.7501, 125), (0.0, 127),
                                        (2.0 ** -140, 1), (3.4e38, 253), (np.inf, 255), (np.nan, 255)])
def test_scale_codes_by_hand(amax, code):
    y = np.zeros((1, 64))
    y[0, 40] = -amax
    assert F.block_scale_codes(y)[0].tolist() == [127, code]


def test_codes_by_hand():
    v = [0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 6.0, -0.25, -0.3, -6.0]
    assert F.nearest_e2m1(v).tolist() == [0, 0, 1, 2, 2, 4, 4, 5, 6, 6, 7, 7, 8, 9, 15]


def test_quantisation_by_hand():
    # the block's largest magnitude 11: 2 * 6 holds it, so the scale is 2 and 11 / 2 = 5.5 rounds to 6
    y = np.zeros((1, 32))
    y[0, :4] = 11, -3, 1, 0.4
    codes, e = F.quantize_fp4(y)
    assert e.tolist() == [[128]] and codes[0, :5].tolist() == [7, 8 + 3, 1, 0, 0]


def test_quantisation_as_the_generator():
    x = np.random.default_rng(3).normal(size=(5, 256)).astype(np.float32)
    codes, e = F.quantize_fp4(x)
    want, want_e = W.quantize_fp4_rows(x)
    # (zeros of either sign are one value)
    assert (e == want_e).all() and (O.decode_e2m1(codes) == O.decode_e2m1(O.unpack_e2m1(want, 256))).all()


def test_values_and_product():
    rng = np.random.default_rng(4)
    a, b = rng.integers(0, 16, (3, 128)), rng.integers(0, 16, (5, 128))
    ea, eb = rng.integers(120, 130, (3, 4)), rng.integers(120, 130, (5, 4))
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    want = np.zeros((3, 5))
    for m in range(3):
        for n in range(5):
            for k in range(128):
                want[m, n] += float(table[a[m, k]] * table[b[n, k]]) * 2.0 ** (int(ea[m, k // 32]) + int(eb[n, k // 32]) - 254)
    got = F.gemm(W.pack_fp4(a.astype(np.uint8)), W.pack_sf(ea.astype(np.uint8)), W.pack_fp4(b.astype(np.uint8)), W.pack_sf(eb.astype(np.uint8)))
    assert np.allclose(got, want, rtol=1e-13)


def _difference(f, x, h=1e-6):
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        v = x[i]
        x[i] = v + h
        up = f()
        x[i] = v - h
        g[i] = (up - f()) / (2 * h)
        x[i] = v
    return g


def test_swiglu_gradient():
    rng = np.random.default_rng(5)
    x, dy = rng.normal(size=(3, 8)) * 2, rng.normal(size=(3, 4))
    assert np.allclose(F.swiglu_backward(x, dy), _difference(lambda: (F.swiglu(x) * dy).sum(), x), atol=1e-8)


def test_balance_by_hand():
    # two live rows: p = (1/2, 1/2, 0) and (1/4, 1/4, 1/2); counts 2, 1, 1 of 4
    x = np.array([[0.0, 0.0, -np.inf], [0.0, 0.0, np.log(2)], [-np.inf, np.nan, -np.inf]])
    loss, counts, live, mean = F.balance_loss(x, [[0, 1], [2, 0], [-1, -1]], coef=0.5)
    assert counts.tolist() == [2, 1, 1] and live == 2 and mean.tolist() == pytest.approx([0.375, 0.375, 0.25])
    assert loss == pytest.approx(0.5 * 3 * (0.5 * 0.375 + 0.25 * 0.375 + 0.25 * 0.25))


def test_balance_of_nothing():
    assert F.balance_loss(np.zeros((0, 3)), np.zeros((0, 1)))[0] == 0
    assert F.balance_loss(np.full((2, 3), -np.inf), [[-1], [-1]])[2] == 0


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_gradient(scoring):
    rng = np.random.default_rng(6)
    x = rng.normal(size=(4, 5)) * 2
    x[2, 1] = -np.inf
    ids = rng.integers(0, 5, (4, 2))
    _, counts, live, _ = F.balance_loss(x, ids, scoring, 0.3)
    got = F.balance_loss_backward(x, counts, live, 1.7, scoring, 0.3)
    want = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        if np.isfinite(x[i]):
            v, h = x[i], 1e-6
            x[i] = v + h
            up = F.balance_loss(x, ids, scoring, 0.3)[0]
            x[i] = v - h
            want[i] = 1.7 * (up - F.balance_loss(x, ids, scoring, 0.3)[0]) / (2 * h)
            x[i] = v
    assert np.allclose(got, want, atol=1e-8)


def test_balance_probabilities_of_small_sigmoids():
    # far below zero the sigmoid is the exponential: shares do not underflow together
    p = F.probabilities([[-800.0, -800.0 + np.log(3), -np.inf]], "sigmoid")
    assert p[0].tolist() == pytest.approx([0.25, 0.75, 0])
