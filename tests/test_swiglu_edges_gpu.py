"""The SwiGLU and its gradient where a gate's exponential, or the products around it, leave the range of FP32.

silu(g) = g / (1 + exp(-g)) is a normal number down to g = -91.9. The exponent of exp(-g) is at most 133 there: it rounds by
2^-18 (half a unit of [64, 128)), its constant's own rounding (2^-26 of itself) adds under 2^-19, so the exponential is off by
1.5 * 2^-18 ln 2 < 2^-17.9 relative, the approximations and products by a few 2^-23 more: NEAR = 2^-17 as for other gates."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.four_bit as F
from test_quantize_fp4_gpu import BF16, NEAR, buffers, check_near, np64

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


def far_gates(first):
    """A row for each four BF16 gates of [first, -40], a block of 32 columns with one gate each, beside `up` of both signs."""
    gates = torch.cat([torch.arange(first, -64, 0.5), torch.arange(-64, -39.9, 0.25)])
    gates = gates[:len(gates) // 4 * 4].view(-1, 4)
    up = torch.randn(len(gates), 128, generator=torch.Generator().manual_seed(1)).clamp_(-3, 3)
    return torch.cat([gates.repeat_interleave(32, 1), up], 1).to("cuda", BF16)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 20, 2.0 ** 100])
def test_small_silu_is_not_zero(lib, scale):
    x = far_gates(-91.5)
    x[:, 128:] *= scale
    q, sf = buffers((), len(x), 128)
    lib.dg_swiglu_quantize_fp4(x, q, sf)
    check_near(F.swiglu(np64(x)), q, sf)


def check_gradient(x, dy, dx):
    """Within the formula's terms, 2^-17 of each, and the rounding to BF16 (of what is below 2^-126 a step of 2^-133)."""
    x64, dy64 = np64(x), np64(dy)
    want = F.swiglu_backward(x64, dy64)
    gate, up = np.split(x64, 2, -1)
    s = 1 / (1 + np.exp(-gate))
    room = np.concatenate([np.abs(dy64 * up * s) * (1 + np.abs(gate)), np.abs(dy64 * gate * s)], -1) * NEAR
    assert (np.abs(np64(dx) - want) <= room + 2.0 ** -8 * np.abs(want) + 2.0 ** -134).all()


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 60])
def test_gradient_of_far_gates_is_not_zero(lib, scale):
    x = far_gates(-91.5)
    dy = (scale * torch.randn(len(x), 128, generator=torch.Generator().manual_seed(2))).to("cuda", BF16)
    dx = torch.full_like(x, 77.0)
    lib.dg_swiglu_backward(x, dy, dx)
    check_gradient(x, dy, dx)


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
