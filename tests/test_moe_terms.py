"""The E4M3 terms of the few-token layer's inner values: the bounds that the header states, and that the check of the
layer with its leading bits cancelled (moe_terms.py) sees each term. Mistakes are planted in the restatement here."""
from __future__ import annotations

import numpy as np
import pytest

import moe_terms as M
from test_moe_gpu import Layer


def _blocks(lo, n=20000):
    """Blocks of 64 of exponents from `lo` up, the largest anywhere in (224, 448] times a power of two."""
    rng = np.random.default_rng(1)
    h = np.exp2(rng.uniform(lo, 7.8, (n, 64))) * rng.choice([-1, 1], (n, 64))
    h[:, 0] = rng.uniform(224.0, 448.0, n) + 2.0 ** -10
    return np.minimum(h, 448.0) * np.exp2(rng.integers(-60, 60, (n, 1)))


@pytest.mark.parametrize("lo", [0, -12, -30])
def test_bounds_of_the_terms(lo):
    h = _blocks(lo)
    err = np.abs(M.as_terms(h) - h)
    top = np.abs(h).max(-1, keepdims=True)
    assert (err <= np.maximum(2.0 ** -16 * np.abs(h), 2.0 ** -29 * top)).all()
    # three would miss even 2^-27 of the largest: 2^-18 / 224 = 2^-25.8
    three = np.abs(M.as_terms(h, M.TERMS[:3]) - h)
    assert lo == 0 or (three > np.maximum(2.0 ** -12 * np.abs(h), 2.0 ** -27 * top)).any()


def test_bound_of_the_smallest_blocks():
    h = np.random.default_rng(2).normal(size=(100, 64)) * np.exp2(np.random.default_rng(3).integers(-149, -100, (100, 1)))
    assert (np.abs(M.as_terms(h) - h) <= np.maximum(2.0 ** -136, 2.0 ** -16 * np.abs(h))).all()


PLANTED = {"as it is": M.TERMS, "without the last": M.TERMS[:3], "without two": M.TERMS[:2], "one alone": M.TERMS[:1],
           "the last as the third": (1.0, 16.0, 256.0, 256.0), "the third as the second": (1.0, 16.0, 16.0, 4096.0),
           "the last too small": (1.0, 16.0, 256.0, 65536.0)}


@pytest.mark.parametrize("planted", PLANTED)
@pytest.mark.parametrize("T, E, k, H, I", [(1, 8, 2, 256, 128), (9, 3, 3, 512, 128), (32, 2, 2, 256, 256), (20, 6, 3, 640, 384)])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_the_check_sees_each_term(planted, T, E, k, H, I, fmt):
    p = Layer(T, E, k, H, I, fmt, seed=T + H)
    part, want = M.cancel(p)
    y = M.bf16(M.layer(p, lambda h: M.as_terms(h, PLANTED[planted])) + want - part)
    assert (M.far(y, part, want) <= M.tolerance(p, part, want)) == (planted == "as it is")
