"""Row strides and sizes at the ends of their range."""
from __future__ import annotations

import ctypes

import pytest
import torch

from test_norm_gpu import lib, make, outputs  # noqa: F401  (lib: the fixture)

pytestmark = pytest.mark.gpu


def odd(row: torch.Tensor) -> torch.Tensor:
    """The row [1, n] again, as the first of rows n + 1 elements apart."""
    wide = torch.full((3, row.shape[1] + 1), float("nan"), dtype=row.dtype, device="cuda")
    wide[:1, :-1] = row
    return wide[:1, :-1]


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_norm_of_one_row_with_any_stride(lib, residual):  # noqa: F811
    H = 384
    x, r, w = make(1, H, residual, torch.bfloat16, seed=1)
    want, got = outputs(lib, 1, H, residual), outputs(lib, 1, H, residual)
    lib.dg_add_rms_norm(x, r, w, 1e-6, **want)
    got["residual_out"] = odd(torch.zeros(1, H, dtype=residual, device="cuda"))
    lib.dg_add_rms_norm(odd(x), odd(r), w, 1e-6, **got)
    assert all(torch.equal(got[k], want[k]) for k in want)
    # and at the C entry
    for k in ("y", "q", "sf", "rstd"):
        got[k].zero_()
    for stride in (0, H + 1):
        d = lib._NormDesc(1, H, stride, stride, stride, lib._TYPES[residual], 0, 1e-6)
        p = [ctypes.c_void_p(t.data_ptr()) for t in (x, r, w, want["residual_out"], got["y"], got["q"], got["sf"], got["rstd"])]
        assert lib.load_library().dg_add_rms_norm(*p, ctypes.byref(d), None) == 0
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E", [60, 256])
def test_router_of_one_row_with_any_stride(lib, dtype, E):  # noqa: F811
    x = torch.randn(1, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(dtype)
    out = []
    for row in (x, odd(x)):
        ids, w, dx = torch.empty(1, 4, dtype=torch.int32, device="cuda"), torch.empty(1, 4, device="cuda"), torch.empty_like(x)
        lib.dg_moe_route(row, ids, w)
        lib.dg_moe_route_backward(row, ids, w, dx)
        out.append((ids, w, dx))
    for stride in (0, E + 1):
        d = lib._RouteDesc(1, E, 4, stride, lib._TYPES[dtype], 0, 1, 1.0)
        ids, w, dx = (torch.empty_like(t) for t in out[0])
        p, pi, pw, pd = (ctypes.c_void_p(t.data_ptr()) for t in (x, ids, w, dx))
        assert lib.load_library().dg_moe_route(p, pi, pw, ctypes.byref(d), None) == 0
        assert lib.load_library().dg_moe_route_backward(p, pi, pw, pd, ctypes.byref(d), None) == 0
        out.append((ids, w, dx))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(o, out[0]))


def test_more_rows_than_an_int_counts_are_refused(lib):  # noqa: F811
    # 2^32 + 3 rows must not pass for 3; they are views of one, so they take no memory
    T = 2 ** 32 + 3
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda").expand(T, 8)
    w, y = torch.ones(8, device="cuda"), x
    with pytest.raises(ValueError, match="size above"):
        lib.dg_add_rms_norm(x, None, w, 1e-6, y=y)
    with pytest.raises(ValueError, match="size above"):
        lib.dg_add_rms_norm_backward(x, x, w, w, None, y, None, w)
    ids, weights = (torch.zeros(1, 2, dtype=d, device="cuda").expand(T, 2) for d in (torch.int32, torch.float32))
    with pytest.raises(ValueError, match="size above"):
        lib.dg_moe_route(x, ids, weights)
    with pytest.raises(ValueError, match="size above"):
        lib.dg_moe_route(x[:1], ids[:1].expand(1, 2)[:, :1].expand(1, T), weights)
