"""The SwiGLU and its gradient where the products around a gate's exponential leave the range of FP32; tolerances as in
test_quantize_fp4_gpu.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.four_bit as F
from test_quantize_fp4_gpu import BF16, NEAR, buffers, np64

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(BF16).min


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    L.dg_get_device_status()
    return L


def check_gradient(x, dy, dx):
    """Within the formula's terms, 2^-17 of each, and the rounding to BF16 (of what is below 2^-126 a step of 2^-133)."""
    x64, dy64 = np64(x), np64(dy)
    want = F.swiglu_backward(x64, dy64)
    gate, up = np.split(x64, 2, -1)
    s = 1 / (1 + np.exp(-gate))
    room = np.concatenate([np.abs(dy64 * up * s) * (1 + np.abs(gate)), np.abs(dy64 * gate * s)], -1) * NEAR
    assert (np.abs(np64(dx) - want) <= room + 2.0 ** -8 * np.abs(want) + 2.0 ** -134).all()


def test_gradient_of_the_lowest_gates(lib):
    # dy * gate is past FP32's range, the gradient is 0: a gate may be masked by the type's lowest value
    x = torch.full((3, 256), 0.5, device="cuda", dtype=BF16)
    x[0, :128], x[1, :64], x[2, ::7] = LOWEST, -1e38, LOWEST
    x[2, 128:] = -4.0
    dy = torch.full((3, 128), 8.0, device="cuda", dtype=BF16)
    dx = torch.full_like(x, 77.0)
    lib.dg_swiglu_backward(x, dy, dx)
    assert dx.isfinite().all()
    far = x[:, :128] < -1000
    assert (dx[:, :128][far] == 0).all() and (dx[:, 128:][far] == 0).all()
    near = torch.cat([~far, ~far], 1)
    want = F.swiglu_backward(np.where(np64(torch.cat([far, far], 1)) > 0, 0, np64(x)), np64(dy))
    got, keep = np64(dx), near.cpu().numpy()
    assert (np.abs(got - want)[keep] <= (2.0 ** -8 + 2 * NEAR) * np.abs(want)[keep]).all()


def test_gradient_of_large_factors(lib):
    # dy * up is past FP32's range, times silu'(gate) it is not
    x = torch.empty(2, 256, device="cuda", dtype=BF16)
    x[:, :128], x[:, 128:] = -60.0, 1e25
    dy = torch.full((2, 128), 1e25, device="cuda", dtype=BF16)
    dy[1] = -1e24
    dx = torch.full_like(x, 77.0)
    lib.dg_swiglu_backward(x, dy, dx)
    check_gradient(x, dy, dx)


def test_lowest_gates_quantise_to_zero(lib):
    x = torch.full((2, 256), 3.0, device="cuda", dtype=BF16)
    x[0, :128], x[1, :128:3] = LOWEST, LOWEST
    q, sf = buffers((), 2, 128)
    lib.dg_swiglu_quantize_fp4(x, q, sf)
    got = F.values(q.cpu().numpy(), sf.cpu().numpy())
    assert (got[0] == 0).all() and (got[1, ::3] == 0).all() and (got[1, 1::3] >= 8).all()
