"""dg_quantize_fp4, dg_swiglu_quantize_fp4 and dg_swiglu_backward against the FP64 oracle.

Codes and scales of plain rows have to be equal: a scale is a power of two, so x times its inverse is exact (or so far
below a half of the least magnitude that it rounds to 0 either way). The SwiGLU is computed in FP32: sigmoid(g) is off by
the rounded exponent of exp (|g| log2 e 2^-24 <= 2^-18 for |g| <= 40), two approximations within 2^-22 and three
roundings, under 2^-17 together; a code may then be the one on the other side of a midpoint that is that near, a scale the
next one where the block's largest magnitude is that near a border. The gradient's factor 1 + g (1 - s) adds terms of up
to 1 + |g|, so it is off by 2^-17 (1 + |g|) of |dy u s|; BF16 rounds to 2^-8."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
import oracle.four_bit as F

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NEAR = 2.0 ** -17


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    L.dg_get_device_status()
    return L


def up4(m):
    return 4 * (-(-m // 4))


def buffers(lead, M, K):
    return (torch.full((*lead, M, K // 2), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((*lead, K // 128, up4(M)), 0x5A5A5A5A, dtype=torch.int32, device="cuda"))


def np64(t):
    return t.double().cpu().numpy()


def check_untouched(q, sf, rows, M):
    """Rows behind the count hold what they held, padding words are 0."""
    assert (q[rows:] == 0xA5).all()
    assert (sf[:, rows:M] == 0x5A5A5A5A).all() and (sf[:, M:] == 0).all()


def check_equal(x, q, sf, rows=None):
    """One group: x [M, K] against its codes and scale words."""
    M, K = x.shape
    rows = M if rows is None else rows
    codes, e = F.quantize_fp4(np64(x)[:rows])
    q, sf = q.cpu().numpy(), sf.cpu().numpy()
    assert (F.scale_bytes(sf, M, K)[:rows] == e).all()
    assert (O.unpack_e2m1(q[:rows], K) == codes).all()
    check_untouched(q, sf, rows, M)


def rows_like(M, K, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, device="cuda", generator=g) * torch.exp(3 * torch.randn(M, K // 32, 1, device="cuda", generator=g)).expand(M, K // 32, 32).reshape(M, K)
    return x.to(dtype)


@pytest.mark.parametrize("M, K", [(1, 128), (1, 7168), (2, 256), (3, 384), (4, 640), (7, 128), (8, 512), (9, 1152), (33, 896), (130, 2048), (257, 1920)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows(lib, M, K, dtype):
    x = rows_like(M, K, dtype, M + K)
    q, sf = buffers((), M, K)
    assert lib.dg_quantize_fp4(x, q, sf) == (q, sf)
    check_equal(x, q, sf)
    assert lib.dg_get_device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_borders(lib, dtype):
    # every value and midpoint of E2M1, of both signs, at scales from the least to the largest; magnitudes at 6 and next to it
    v = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
    block = np.concatenate([v, -v, [6, -6]])
    exps = np.concatenate([np.arange(-130, 126, 3), [125]])
    x = np.ldexp(block[None], exps[:, None])
    x = np.concatenate([x, np.ldexp(np.nextafter(np.float32(block), np.float32(9)).astype(np.float64)[None], exps[:, None])])
    x = torch.from_numpy(np.tile(x, (1, 4)).astype(np.float32)).cuda().to(dtype)
    x = torch.where(x.isfinite(), x, 0)
    q, sf = buffers((), *x.shape)
    lib.dg_quantize_fp4(x, q, sf)
    check_equal(x, q, sf)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zeros_and_subnormals(lib, dtype):
    x = torch.zeros(5, 256, device="cuda", dtype=dtype)
    x[1, ::2] = -0.0
    x[2] = 1e-40                                   # subnormal in FP32 and in BF16
    x[3, 5], x[3, 200] = torch.finfo(dtype).max, -torch.finfo(dtype).max
    x[4, 0] = torch.finfo(dtype).tiny
    q, sf = buffers((), 5, 256)
    lib.dg_quantize_fp4(x, q, sf)
    check_equal(x, q, sf)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_that_are_not_finite(lib, dtype):
    x = rows_like(6, 384, dtype, 1)
    x[0, 3], x[1, 40], x[2, 383], x[3, 128:160] = float("nan"), float("inf"), -float("inf"), float("nan")
    q, sf = buffers((), 6, 384)
    lib.dg_quantize_fp4(x, q, sf)
    check_equal(x, q, sf)                          # the block's scale is 255, its neighbours' are their own
    assert F.scale_bytes(sf.cpu().numpy(), 6, 384)[0, :2].tolist()[0] == 255


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows_and_groups(lib, dtype):
    store = rows_like(3 * 40, 640, dtype, 2).view(3, 40, 640)
    x = store[:, 3:24:4, 128:512]                  # rows 2560 elements apart
    q, sf = buffers((3,), *x.shape[1:])
    lib.dg_quantize_fp4(x, q, sf)
    for g in range(3):
        check_equal(x[g], q[g], sf[g])
    one = store[1, 7:8, 256:512]
    q, sf = buffers((), 1, 256)
    lib.dg_quantize_fp4(one, q, sf)
    check_equal(one, q, sf)
    lib.dg_quantize_fp4(store[:1, :5, :256], *(buffers((1,), 5, 256)))
    broadcast = store[0, :1, :256].expand(6, 256)  # every row the same memory
    q, sf = buffers((), 6, 256)
    lib.dg_get_device_status()
    with pytest.raises(lib.DGError):               # rows that overlap are refused
        lib.dg_quantize_fp4(broadcast, q, sf)


@pytest.mark.parametrize("counts", [[0, 5, 37, 1], [37, 37, 37, 37], [0, 0, 0, 0], [8, 9, 16, 36]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masked_rows(lib, counts, dtype):
    x = rows_like(4 * 37, 256, dtype, 3).view(4, 37, 256)
    for g, c in enumerate(counts):
        x[g, c:] = float("nan")                    # not read as values
    q, sf = buffers((4,), 37, 256)
    lib.dg_quantize_fp4(x, q, sf, masked_m=torch.tensor(counts, dtype=torch.int32, device="cuda"))
    for g, c in enumerate(counts):
        check_equal(x[g], q[g], sf[g], rows=c)
    assert lib.dg_get_device_status() == 0


def test_counts_out_of_range(lib):
    x = rows_like(2 * 9, 128, BF16, 4).view(2, 9, 128)
    q, sf = buffers((2,), 9, 128)
    lib.dg_quantize_fp4(x, q, sf, masked_m=torch.tensor([-3, 12], dtype=torch.int32, device="cuda"))
    assert lib.dg_get_device_status() == 6
    check_equal(x[0], q[0], sf[0], rows=0)
    check_equal(x[1], q[1], sf[1], rows=9)


def test_rows_past_32_bits(lib):
    ld = 2 ** 31 + 128                             # the second and third row begin past 2^31 and 2^32 elements
    store = torch.empty(2 * ld + 256, dtype=BF16, device="cuda")
    x = store.as_strided((3, 256), (ld, 1))
    x.copy_(rows_like(3, 256, BF16, 5))
    q, sf = buffers((), 3, 256)
    lib.dg_quantize_fp4(x, q, sf)
    check_equal(x, q, sf)


# --------------------------------------------------------------------------------------
# SwiGLU
# --------------------------------------------------------------------------------------

def check_near(y, q, sf, rows=None):
    """One group's codes and scales of values that may be NEAR off."""
    M, K = y.shape
    rows = M if rows is None else rows
    q, sf = q.cpu().numpy(), sf.cpu().numpy()
    check_untouched(q, sf, rows, M)
    y, e = y[:rows], F.scale_bytes(sf, M, K)[:rows].astype(np.int64)
    low, high = F.block_scale_codes(y * (1 - NEAR)), F.block_scale_codes(y * (1 + NEAR))
    assert ((low <= e) & (e <= high)).all()
    v = y * np.exp2(127.0 - np.repeat(e, 32, -1))
    got = O.decode_e2m1(O.unpack_e2m1(q[:rows], K))
    gap = np.abs(np.abs(v)[..., None] - F.MAGNITUDES).min(-1)
    assert (np.abs(got - v) <= gap + 2 * NEAR * np.abs(v)).all()


def gates(M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 4 * torch.randn(M, 2 * K, device="cuda", generator=g)
    return x.clamp_(-40, 40).to(BF16)


@pytest.mark.parametrize("M, K", [(1, 128), (1, 2048), (5, 256), (9, 384), (66, 896)])
def test_swiglu(lib, M, K):
    x = gates(M, K, M + K)
    q, sf = buffers((), M, K)
    lib.dg_swiglu_quantize_fp4(x, q, sf)
    check_near(F.swiglu(np64(x)), q, sf)
    assert lib.dg_get_device_status() == 0


def test_swiglu_masked_and_strided(lib):
    counts = [0, 21, 7]
    store = gates(3 * 42, 256, 7).view(3, 42, 512)
    x = store[:, ::2]
    for g, c in enumerate(counts):
        x[g, c:] = float("nan")
    q, sf = buffers((3,), 21, 256)
    lib.dg_swiglu_quantize_fp4(x, q, sf, masked_m=torch.tensor(counts, dtype=torch.int32, device="cuda"))
    for g, c in enumerate(counts):
        check_near(F.swiglu(np64(x[g])), q[g], sf[g], rows=c)


def test_swiglu_far_gates(lib):
    # exp(-g) overflows and vanishes: y is 0 and g u
    x = torch.zeros(2, 256, device="cuda", dtype=BF16)
    x[0, :128], x[1, :128], x[:, 128:] = -200.0, 200.0, 0.5
    q, sf = buffers((), 2, 128)
    lib.dg_swiglu_quantize_fp4(x, q, sf)
    got = F.values(q.cpu().numpy(), sf.cpu().numpy())
    assert (got[0] == 0).all() and (np.abs(got[1] - 100) <= 100 / 8).all()


def test_swiglu_not_finite(lib):
    x = gates(3, 128, 8)
    x[0, 5], x[1, 128 + 40], x[2, 127] = float("nan"), float("inf"), float("nan")
    q, sf = buffers((), 3, 128)
    lib.dg_swiglu_quantize_fp4(x, q, sf)
    e = F.scale_bytes(sf.cpu().numpy(), 3, 128)
    assert [int(e[0, 0]), int(e[1, 1]), int(e[2, 3])] == [255] * 3 and (e == 255).sum() == 3


@pytest.mark.parametrize("lead, M, K, counts", [((), 1, 128, None), ((), 5, 384, None), ((), 67, 1152, None), ((3,), 10, 256, [0, 10, 3]), ((2,), 1, 640, [1, 0])])
@pytest.mark.parametrize("in_place", [False, True])
def test_swiglu_gradient(lib, lead, M, K, counts, in_place):
    x = gates(M * int(np.prod(lead)), K, 9).view(*lead, M, 2 * K)
    dy = torch.randn(*lead, M, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(10)).to(BF16)
    before = x.clone()
    dx = x if in_place else torch.full_like(x, 77.0)
    masked = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    assert lib.dg_swiglu_backward(x, dy, dx, masked_m=masked) is dx
    x64, dy64 = np64(before), np64(dy)
    want = F.swiglu_backward(x64, dy64)
    gate, u = np.split(x64, 2, -1)
    s = 1 / (1 + np.exp(-gate))
    room = np.concatenate([np.abs(dy64 * u * s) * (1 + np.abs(gate)), np.abs(dy64 * gate * s)], -1) * NEAR
    kept = np.ones((*lead, M, 1), bool) if counts is None else (np.arange(M)[None] < np.array(counts)[:, None])[..., None]
    got = np64(dx)
    old = x64 if in_place else 77.0
    assert (np.abs(got - np.where(kept, want, old)) <= np.where(kept, room + 2.0 ** -8 * np.abs(want) + 2.0 ** -134, 0)).all()


def test_swiglu_gradient_of_strided_rows(lib):
    store = gates(20, 256, 11).view(20, 512)
    x, dy = store[3:17:3], torch.randn(5, 256, device="cuda").to(BF16)
    dx, same = torch.empty(5, 512, device="cuda", dtype=BF16), torch.empty(5, 512, device="cuda", dtype=BF16)
    lib.dg_swiglu_backward(x, dy, dx)
    lib.dg_swiglu_backward(x.contiguous(), dy, same)
    assert torch.equal(dx, same)
