"""Pins of the layer oracle (oracle/layers.py): hand-worked values, central differences of its own
forward formulas for the gradients, and an independent torch form of the mixture-of-experts layer."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.layers as L
import workloads as W


def test_norm_by_hand():
    # s = (3, 4): mean square 12.5; weight (1, 2)
    s, rstd, y = L.add_rms_norm([[1.0, 1.0]], [[2.0, 3.0]], [1.0, 2.0], 0.0)
    assert s.tolist() == [[3.0, 4.0]]
    assert rstd[0] == pytest.approx(12.5 ** -0.5)
    assert y[0].tolist() == pytest.approx([3 * 12.5 ** -0.5, 8 * 12.5 ** -0.5])


@pytest.mark.parametrize("amax, code", [(448.0, 127), (448.0001, 128), (224.0, 126), (1.0, 119), (0.875, 118), (0.8751, 119),
                                        (0.0, 127), (2.0 ** -130, 1), (3e38, 247)])
def test_scale_codes_by_hand(amax, code):
    y = np.zeros((1, 128))
    y[0, 77] = -amax
    assert L.group_scale_codes(y)[0, 0] == code


def test_scale_codes_ignore_what_is_not_finite():
    y = np.full((1, 128), 2.0)
    y[0, 0], y[0, 1], y[0, 2] = np.nan, np.inf, -np.inf
    assert L.group_scale_codes(y)[0, 0] == 120


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


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    s, w, dy, ds = rng.normal(size=(3, 9)), rng.normal(size=9), rng.normal(size=(3, 9)), rng.normal(size=(3, 9))
    eps = 1e-2

    def f():
        v, _, y = L.add_rms_norm(s, None, w, eps)
        return (dy * y).sum() + (ds * v).sum()

    d, dw = L.add_rms_norm_backward(dy, s, w, L.add_rms_norm(s, None, w, eps)[1], ds)
    # central differences of step 1e-6: their own error is about 1e-9
    np.testing.assert_allclose(d, _difference(f, s), atol=1e-7)
    np.testing.assert_allclose(dw, _difference(f, w), atol=1e-7)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(scoring, renormalize):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(4, 7))
    x[1, 3] = x[1, 5] = -np.inf
    ids, _ = L.moe_route(x, 3, scoring, renormalize, 1.5)
    dw = rng.normal(size=(4, 3))
    live = np.where(np.isfinite(x), x, 0.0)

    def f():
        row = np.where(np.isfinite(x), live, -np.inf)
        again, w = L.moe_route(row, 3, scoring, renormalize, 1.5)
        assert (again == ids).all()
        return (w * dw).sum()

    want = _difference(f, live) * np.isfinite(x)
    np.testing.assert_allclose(L.moe_route_backward(x, ids, dw, scoring, renormalize, 1.5), want, atol=1e-7)


def test_route_by_hand():
    inf = np.inf
    ids, w = L.moe_route([[1.0, 3.0, 3.0, -inf], [-inf, np.nan, -inf, 2.0], [-inf] * 4], 2)
    assert ids.tolist() == [[1, 2], [3, -1], [-1, -1]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]]
    _, w = L.moe_route([[0.0, 0.0, 0.0]], 1, "softmax", False, 3.0)
    assert w[0, 0] == pytest.approx(1.0)
    _, w = L.moe_route([[0.0, -2.0]], 1, "sigmoid", False)
    assert w[0, 0] == pytest.approx(0.5)


@pytest.mark.parametrize("b_format", ["e4m3", "e2m1"])
def test_moe_layer_against_an_independent_form(b_format):
    rng = np.random.default_rng(3)
    T, E, k, H, I = 3, 4, 2, 256, 128
    xf = rng.normal(size=(T, H)).astype(np.float32)
    x, ex = W.quantize_rows(xf)
    quant = W.quantize_blocks if b_format == "e4m3" else W.quantize_fp4_rows
    f13 = rng.normal(size=(E, 2 * I, H)).astype(np.float32) / 16
    f2 = rng.normal(size=(E, H, I)).astype(np.float32) / 16
    q13, q2 = [quant(m) for m in f13], [quant(m) for m in f2]
    ids = np.array([[0, 3], [1, -1], [2, 2]])
    w = rng.random((T, k))
    got = L.moe_layer(x, W.pack_sf(ex), np.stack([q[0] for q in q13]), np.stack([W.pack_sf(q[1]) if b_format == "e4m3" else _rows(q[1]) for q in q13]),
                      np.stack([q[0] for q in q2]), np.stack([W.pack_sf(q[1]) if b_format == "e4m3" else _rows(q[1]) for q in q2]), ids, w, None, b_format)
    # the same layer from the unquantised values: quantisation to 3 (1) mantissa bits is all that differs
    t = torch.from_numpy
    want = np.zeros((T, H))
    for i in range(T):
        for j in range(k):
            if ids[i, j] >= 0:
                z = t(f13[ids[i, j]]).double() @ t(xf[i]).double()
                h = torch.nn.functional.silu(z[:I]) * z[I:]
                want[i] += w[i, j] * (t(f2[ids[i, j]]).double() @ h).numpy()
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    # each of the three products carries the rounding of its operands: at most 2^-4 relative per element
    # for E4M3, 1/4 for E2M1, averaging out over the terms
    assert rel < (0.12 if b_format == "e4m3" else 0.5), rel


def _rows(exps):
    """[N, K/32] exponents -> packed words [K/128, ceil4(N)]."""
    N, kb = exps.shape
    out = np.zeros((kb // 4, 4 * (-(-N // 4)), 4), np.uint8)
    out[:, :N] = exps.reshape(N, kb // 4, 4).transpose(1, 0, 2)
    return out.reshape(kb // 4, -1).view(np.int32)
