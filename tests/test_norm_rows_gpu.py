"""The norm and its gradient where a team of warps takes many rows in turn: few SMs, so that copies of the next row run
under the row worked on, in a ring of two rows or (the gradient of wide FP32 rows) of one, and dw gathers in registers.
Tolerances as in test_norm_gpu.py; a row's own outputs have the same bits whichever team takes it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.layers as OL
from test_norm_gpu import BF16_REL, F32_REL, check, f64, lib, make, outputs  # noqa: F401  (lib: the fixture)

pytestmark = pytest.mark.gpu

TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)]


@pytest.fixture
def two_sms(lib):  # noqa: F811
    lib.dg_set_num_sms(2)
    yield lib
    lib.dg_set_num_sms(0)


@pytest.mark.parametrize("T, H", [(1001, 128), (613, 512), (301, 640), (203, 1152), (150, 1536), (97, 2176), (50, 4096), (33, 7168), (21, 16384)])
@pytest.mark.parametrize("residual, weight", TYPES)
def test_forward(two_sms, T, H, residual, weight):
    L = two_sms
    x, r, w = make(T, H, residual, weight, seed=T + H)
    o = outputs(L, T, H, residual)
    L.dg_add_rms_norm(x, r, w, 1e-6, **o)
    check(L, x, r, w, 1e-6, o)
    L.dg_set_num_sms(0)
    again = outputs(L, T, H, residual)
    L.dg_add_rms_norm(x, r, w, 1e-6, **again)
    assert all(torch.equal(o[k], again[k]) for k in o)
    L.dg_set_num_sms(2)
    xs, rs = x.clone(), r.clone()            # in place, the next row's copies under way
    L.dg_add_rms_norm(xs, rs, w, 1e-6, residual_out=rs, y=xs)
    assert torch.equal(rs, o["residual_out"]) and torch.equal(xs, o["y"])


@pytest.mark.parametrize("T, H", [(1001, 8), (999, 136), (613, 512), (301, 1000), (203, 1152), (150, 1536), (97, 2048), (64, 4096), (33, 7168),
                                  (31, 10240), (29, 10248), (21, 16384)])
@pytest.mark.parametrize("residual, weight", TYPES)
def test_gradient(two_sms, T, H, residual, weight):
    L = two_sms
    g = torch.Generator(device="cuda").manual_seed(T + H)
    s, ds = [(k * torch.randn(T, H, device="cuda", generator=g)).to(residual) for k in (3, 1)]
    dy = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    w = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(weight)
    rstd = (s.float().square().mean(-1) + 1e-6).rsqrt()

    def run(dy=dy, ds=ds, dx=None, dr=None):
        dx = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda") if dx is None else dx
        dr = torch.full((T, H), float("nan"), dtype=residual, device="cuda") if dr is None else dr
        dw = torch.full((H,), float("nan"), device="cuda")
        L.dg_add_rms_norm_backward(dy, s, w, rstd, ds, dx, dr, dw)
        return dx, dr, dw

    dx, dr, dw = run()
    want, want_w = OL.add_rms_norm_backward(f64(dy), f64(s), f64(w), f64(rstd), f64(ds))
    xhat = f64(s) * f64(rstd)[:, None]
    gy = f64(dy) * f64(w)
    tol = F32_REL * (f64(rstd)[:, None] * (np.abs(gy) + np.abs(xhat) * np.mean(np.abs(gy * xhat), -1, keepdims=True)) + np.abs(f64(ds)))
    assert (np.abs(f64(dx) - want) <= BF16_REL * np.abs(want) + 2 * tol).all()
    rel = BF16_REL if residual == torch.bfloat16 else 2.0 ** -24
    assert (np.abs(f64(dr) - want) <= rel * np.abs(want) + 2 * tol).all()
    assert (np.abs(f64(dw) - want_w) <= (T + 64) * 2.0 ** -24 * np.abs(f64(dy) * xhat).sum(0)).all()
    dyc, dsc = dy.clone(), ds.clone()        # in place
    again = run(dyc, dsc, dyc, dsc)
    assert torch.equal(dyc, dx) and torch.equal(dsc, dr) and torch.equal(again[2], dw)
    L.dg_set_num_sms(0)
    again = run()
    assert torch.equal(again[0], dx) and torch.equal(again[1], dr)
    assert (np.abs(f64(again[2]) - want_w) <= (T + 64) * 2.0 ** -24 * np.abs(f64(dy) * xhat).sum(0)).all()
