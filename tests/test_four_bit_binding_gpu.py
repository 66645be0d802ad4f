"""Tensors that the Python binding of the four-bit operators and of the balance loss refuses."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as lib
    lib.load_library()
    return lib


def new(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("name, per", [("dg_quantize_fp4", 1), ("dg_swiglu_quantize_fp4", 2)])
def test_quantisers(L, name, per):
    call = getattr(L, name)
    x, q, sf = new(6, 256 * per), new(6, 128, dtype=U8), new(2, 8, dtype=I32)
    call(x, q, sf)
    call(new(0, 256 * per), new(0, 128, dtype=U8), new(2, 0, dtype=I32))
    bad = [(x.half(), q, sf), (x.cpu(), q, sf), (x[0], q, sf), (x[:, :-1], q, sf), (x[:, :128 * per - 2], q, sf), (new(256 * per, 6).t(), q, sf),
           (x, q[:, :64], sf), (x, q.int(), sf), (x, q[:5], sf), (x, q, sf[:, :4]), (x, q, sf[:1]), (x, q, sf.float()), (x, q.cpu(), sf),
           (x, new(6, 256, dtype=U8)[:, ::2], sf)]
    for args in bad:
        with pytest.raises(ValueError):
            call(*args)
    for counts in (new(1, dtype=I32), new(2, dtype=I32)):
        with pytest.raises(ValueError):
            call(x, q, sf, masked_m=counts)                      # no groups
    with pytest.raises(ValueError):
        call(x[None], q[None], sf[None], masked_m=new(2, dtype=I32))
    with pytest.raises(L.DGError):
        call(new(6, 256 * per + 4)[:, :256 * per], q, sf)        # rows that begin at no multiple of 16 bytes


def test_swiglu_gradient(L):
    x, dy = new(6, 512), new(6, 256)
    L.dg_swiglu_backward(x, dy, new(6, 512))
    for args in ((x, dy[:, :128], new(6, 512)), (x, dy, new(6, 256)), (x.float(), dy, new(6, 512)), (x, dy.float(), new(6, 512)), (x, dy, new(6, 1024)[:, ::2])):
        with pytest.raises(ValueError):
            L.dg_swiglu_backward(*args)


def test_products(L):
    a, b, sfa, sfb, d = new(6, 128, dtype=U8), new(32, 128, dtype=U8), new(2, 8, dtype=I32), new(2, 32, dtype=I32), new(6, 32)
    L.dg_fp4_gemm_nt(a, sfa, b, sfb, None, d)
    L.dg_fp4_gemm_nt(a, sfa, b, sfb, d, d)
    L.dg_fp4_gemm_nt(a[:0], new(2, 0, dtype=I32), b, sfb, None, d[:0])
    for args in ((a[:, :64], sfa, b, sfb, None, d), (a, sfa, b, sfb, d[:5], d), (a, sfa, b, sfb, None, d.float()), (a, sfa[:1], b, sfb, None, d),
                 (a, sfa, b, sfb[:, :16], None, d), (a.cpu(), sfa, b, sfb, None, d), (a, sfa, b.int(), sfb, None, d), (a[None], sfa, b, sfb, None, d)):
        with pytest.raises(ValueError):
            L.dg_fp4_gemm_nt(*args)
    three, index, counts = b[None].repeat(3, 1, 1), new(6, dtype=I32), new(3, dtype=I32)
    sf3 = sfb[None].repeat(3, 1, 1)
    L.dg_m_grouped_fp4_gemm_nt_contiguous(a, sfa, three, sf3, d, index)
    for args in ((a, sfa, b, sf3, d, index), (a, sfa, three, sfb, d, index), (a, sfa, three, sf3, d, index[:5]), (a, sfa, three, sf3, d, index.long())):
        with pytest.raises(ValueError):
            L.dg_m_grouped_fp4_gemm_nt_contiguous(*args)
    a3, sa3, d3 = a[None].repeat(3, 1, 1), sfa[None].repeat(3, 1, 1), d[None].repeat(3, 1, 1)
    L.dg_m_grouped_fp4_gemm_nt_masked(a3, sa3, three, sf3, d3, counts)
    for args in ((a, sa3, three, sf3, d3, counts), (a3, sa3[:2], three, sf3, d3, counts), (a3, sa3, three[:2], sf3, d3, counts), (a3, sa3, three, sf3, d3, counts[:2])):
        with pytest.raises(ValueError):
            L.dg_m_grouped_fp4_gemm_nt_masked(*args)
    assert L.dg_get_device_status() == 0


def test_balance(L):
    x, ids = new(5, 12, dtype=torch.float32), new(5, 2, dtype=I32)
    out = lambda: [new(12, dtype=I32), new(1, dtype=I32), new(12, dtype=torch.float32), new(1, dtype=torch.float32)]  # noqa: E731
    L.dg_moe_balance_loss(x, ids, *out())
    for i in range(4):
        wrong = out()
        wrong[i] = wrong[i][:-1]
        with pytest.raises(ValueError):
            L.dg_moe_balance_loss(x, ids, *wrong)
    for args in ((x.half(), ids), (x, ids.long()), (x, ids[:4]), (x[0], ids)):
        with pytest.raises(ValueError):
            L.dg_moe_balance_loss(*args, *out())
    with pytest.raises(ValueError):
        L.dg_moe_balance_loss(x, ids, *out(), scoring="other")
    with pytest.raises(L.DGError):
        L.dg_moe_balance_loss(x, ids, *out(), coef=float("nan"))
    counts, live, _, one = out()
    L.dg_moe_balance_loss_backward(x, counts, live, one, new(5, 12, dtype=torch.float32))
    for args in ((x, counts[:11], live, one, x), (x, counts, live, one, x.bfloat16()), (x, counts, live.float(), one, x)):
        with pytest.raises(ValueError):
            L.dg_moe_balance_loss_backward(*args)
    with pytest.raises(ValueError):
        L.dg_moe_balance_loss_backward(x, counts, live, one, new(5, 12, dtype=torch.float32), base=x.bfloat16())
