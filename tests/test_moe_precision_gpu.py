"""The few-token layer to the last bits of its sums: an addend cancels the leading ones (moe_terms.py derives how far the
rest may be), and single inner values stand beside much larger ones of their block."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_terms as M
import workloads as W
from test_moe_gpu import SHAPES, Layer, lib  # noqa: F401  (lib: the fixture)
from test_moe_parts_gpu import CUT

pytestmark = pytest.mark.gpu


def close(p, y, part, want):
    return M.far(y.double().cpu().numpy(), part, want) <= M.tolerance(p, part, want)


@pytest.mark.parametrize("T, E, k, H, I", SHAPES + CUT + [(32, 3, 1, 384, 256), (25, 2, 1, 384, 256), (32, 40, 8, 1536, 640), (7, 100, 9, 512, 640)])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_leading_bits_cancelled(lib, T, E, k, H, I, fmt):  # noqa: F811
    p = Layer(T, E, k, H, I, fmt, seed=T * 37 + E + I)
    part, want = M.cancel(p)
    assert close(p, p.run(lib), part, want)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_empty_slots_and_duplicates_cancelled(lib, fmt):  # noqa: F811
    p = Layer(12, 5, 4, 256, 128, fmt, seed=7)
    p.ids[0] = -1
    p.ids[1] = [3, 3, -1, 3]
    p.ids[2, 1] = -1
    p.weights[3] = 0
    p.weights[4] = [-1.0, 3.0, 0.0, -2.0]
    part, want = M.cancel(p)
    assert close(p, p.run(lib), part, want)


@pytest.mark.parametrize("T, E, k, H, I", [(11, 6, 3, 512, 384), (20, 6, 3, 2304, 1152)])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_other_numbers_of_sms_cancelled(lib, T, E, k, H, I, fmt):  # noqa: F811
    p = Layer(T, E, k, H, I, fmt, seed=11)
    part, want = M.cancel(p)
    try:
        for sms in (1, 5, 64, 151):
            lib.dg_set_num_sms(sms)
            assert close(p, p.run(lib), part, want), sms
    finally:
        lib.dg_set_num_sms(0)


def test_small_values_beside_large_ones(lib):  # noqa: F811
    # gate row j times x is g_j, up row j times x is u_j times a power of two of the token's, and W2 is the identity: y is h
    # itself. One value of every 64 is 2^25 to 2^36 times the others. exp and the few products of h are within 2^-18.
    T, H, I = 3, 128, 128
    p = Layer(T, 2, 1, H, I, "e4m3", seed=21, c=False)
    rng = np.random.default_rng(21)
    code = lambda v: torch.from_numpy(np.asarray(v, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()  # noqa: E731
    p.x[:], p.w13[:], p.w2[:] = 0, 0, 0
    p.x[:, 0], p.x[:, 1] = code(1.0), code([1.0, 2.0, 0.25])
    p.sfx, p.sf13, p.sf2 = (np.full_like(v, 0x7F7F7F7F) for v in (p.sfx, p.sf13, p.sf2))
    g, u = rng.uniform(-17, -12, (2, I)), rng.uniform(0.25, 4, (2, I)) * rng.choice([-1, 1], (2, I))
    g[:, ::64], u[:, ::64] = 20.0, rng.uniform(230, 448, (2, I // 64))
    p.w13[:, :I, 0], p.w13[:, I:, 1] = code(g), code(u)
    p.w2[:, np.arange(I), np.arange(I)] = code(1.0)
    want = M.layer(p)
    top = np.repeat(np.abs(want).reshape(T, I // 64, 64).max(-1), 64, -1)
    got = p.run(lib).double().cpu().numpy()
    bound = np.maximum(2.0 ** -16 * np.abs(want), 2.0 ** -29 * top) + (2.0 ** -18 + 2.0 ** -8) * np.abs(want)
    assert (np.abs(got - want) <= bound).all()
    assert (np.abs(want) < 2.0 ** -24 * top).sum() > 100
    # what three terms would leave of them: the bound is not met by far
    three = np.abs(M.as_terms(want, M.TERMS[:3]) - want)
    assert (three > 3 * bound).any()
