"""Arguments that the four-bit operators and the balance loss refuse before they touch the device (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest

P = ctypes.c_void_p
X = P(0x10000)           # never dereferenced: validation fails first
ODD = P(0x10008)
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    from fp8_gemm_nt_gb300 import build
    build.build()
    import fp8_gemm_nt_gb300 as pkg
    pkg.load_library()
    return pkg


def quantize(L, name, x=X, masked=None, q=X, sf=X, G=1, M=4, K=256, ldx=512, ldg=0, xt=0):
    d = L._RowsDesc(G, M, K, ldx, ldg, xt)
    return getattr(L.load_library(), name)(x, masked, q, sf, ctypes.byref(d), None)


@pytest.mark.parametrize("name", ["dg_quantize_fp4", "dg_swiglu_quantize_fp4"])
@pytest.mark.parametrize("status, over", [
    (INVALID, dict(x=None)), (INVALID, dict(q=None)), (INVALID, dict(sf=None)), (INVALID, dict(G=0)), (INVALID, dict(G=-1)), (INVALID, dict(M=-1)),
    (INVALID, dict(K=0)), (INVALID, dict(K=192)), (INVALID, dict(K=-128)), (INVALID, dict(xt=2)), (INVALID, dict(xt=-1)), (INVALID, dict(ldx=128)),
    (INVALID, dict(ldx=0)), (MISALIGNED, dict(x=ODD)), (MISALIGNED, dict(q=ODD)), (MISALIGNED, dict(sf=ODD)), (MISALIGNED, dict(masked=P(0x10002))),
    (MISALIGNED, dict(ldx=516)), (MISALIGNED, dict(G=2, ldg=2052)), (UNSUPPORTED, dict(K=2 ** 30 + 128, ldx=2 ** 32)), (UNSUPPORTED, dict(M=BIG)),
    (UNSUPPORTED, dict(G=BIG, M=2 ** 30)), (OK, dict(M=0)), (OK, dict(M=0, x=None, q=None, sf=None))])
def test_quantize(L, name, status, over):
    assert quantize(L, name, **over) == status


def test_swiglu_takes_bf16(L):
    assert quantize(L, "dg_swiglu_quantize_fp4", xt=1) == INVALID
    assert quantize(L, "dg_swiglu_quantize_fp4", K=2 ** 29 + 128, ldx=2 ** 32) == UNSUPPORTED


def swiglu_gradient(L, x=X, dy=X, masked=None, dx=X, G=1, M=4, K=256, ldx=512, ldg=0, xt=0):
    d = L._RowsDesc(G, M, K, ldx, ldg, xt)
    return L.load_library().dg_swiglu_backward(x, dy, masked, dx, ctypes.byref(d), None)


@pytest.mark.parametrize("status, over", [
    (INVALID, dict(x=None)), (INVALID, dict(dy=None)), (INVALID, dict(dx=None)), (INVALID, dict(xt=1)), (INVALID, dict(K=100)), (INVALID, dict(ldx=256)),
    (MISALIGNED, dict(dy=ODD)), (MISALIGNED, dict(dx=ODD)), (MISALIGNED, dict(ldx=1020)), (OK, dict(M=0))])
def test_swiglu_gradient(L, status, over):
    assert swiglu_gradient(L, **over) == status


@pytest.mark.parametrize("name", ["dg_quantize_fp4", "dg_swiglu_quantize_fp4", "dg_swiglu_backward"])
def test_without_sizes(L, name):
    assert getattr(L.load_library(), name)(X, X, X, X, None, None) == INVALID


def balance(L, logits=X, ids=X, counts=X, live=X, mean=X, loss=X, T=4, E=16, k=2, ld=16, lt=1, scoring=0, coef=1.0):
    d = L._BalanceDesc(T, E, k, ld, lt, scoring, coef)
    return L.load_library().dg_moe_balance_loss(logits, ids, counts, live, mean, loss, ctypes.byref(d), None)


@pytest.mark.parametrize("status, over", [
    (INVALID, dict(logits=None)), (INVALID, dict(ids=None)), (INVALID, dict(counts=None)), (INVALID, dict(live=None)), (INVALID, dict(mean=None)),
    (INVALID, dict(loss=None)), (INVALID, dict(T=-1)), (INVALID, dict(E=0)), (INVALID, dict(k=0)), (INVALID, dict(ld=15)), (INVALID, dict(lt=2)),
    (INVALID, dict(scoring=2)), (INVALID, dict(coef=float("nan"))), (INVALID, dict(coef=float("inf"))), (UNSUPPORTED, dict(E=1025, ld=1025)),
    (UNSUPPORTED, dict(k=33)), (UNSUPPORTED, dict(T=2 ** 30, k=4)), (MISALIGNED, dict(logits=P(0x10002))), (MISALIGNED, dict(lt=0, logits=P(0x10001))),
    (MISALIGNED, dict(ids=P(0x10002))), (MISALIGNED, dict(counts=P(0x10001))), (MISALIGNED, dict(live=P(0x10002))), (MISALIGNED, dict(mean=P(0x10002))),
    (MISALIGNED, dict(loss=P(0x10002)))])
def test_balance(L, status, over):
    assert balance(L, **over) == status


def balance_gradient(L, logits=X, counts=X, live=X, dloss=X, base=X, dx=X, T=4, E=16, ld=16, lt=1, scoring=0, coef=1.0):
    d = L._BalanceDesc(T, E, 0, ld, lt, scoring, coef)
    return L.load_library().dg_moe_balance_loss_backward(logits, counts, live, dloss, base, dx, ctypes.byref(d), None)


@pytest.mark.parametrize("status, over", [
    (INVALID, dict(logits=None)), (INVALID, dict(counts=None)), (INVALID, dict(live=None)), (INVALID, dict(dloss=None)), (INVALID, dict(dx=None)),
    (INVALID, dict(T=-1)), (INVALID, dict(scoring=-1)), (INVALID, dict(ld=3)), (UNSUPPORTED, dict(E=2000, ld=2000)), (MISALIGNED, dict(base=P(0x10002))),
    (MISALIGNED, dict(dx=P(0x10001))), (MISALIGNED, dict(dloss=P(0x10002))), (OK, dict(T=0)), (OK, dict(T=0, logits=None, counts=None, dx=None))])
def test_balance_gradient(L, status, over):
    assert balance_gradient(L, **over) == status


def gemm(L, a=X, sfa=X, b=X, sfb=X, c=None, d=X, M=4, N=64, K=256):
    return L.load_library().dg_fp4_gemm_nt(a, sfa, b, sfb, c, d, M, N, K, None)


def masked(L, a=X, sfa=X, b=X, sfb=X, d=X, counts=X, G=2, M=4, N=64, K=256):
    return L.load_library().dg_m_grouped_fp4_gemm_nt_masked(a, sfa, b, sfb, d, counts, G, M, N, K, None)


def contiguous(L, a=X, sfa=X, b=X, sfb=X, d=X, counts=X, G=2, M=4, N=64, K=256):
    return L.load_library().dg_m_grouped_fp4_gemm_nt_contiguous(a, sfa, b, sfb, d, counts, M, N, K, G, None)


GEMM = [(INVALID, dict(a=None)), (INVALID, dict(sfa=None)), (INVALID, dict(b=None)), (INVALID, dict(sfb=None)), (INVALID, dict(d=None)), (INVALID, dict(M=-1)),
        (INVALID, dict(N=0)), (INVALID, dict(N=24)), (INVALID, dict(K=0)), (INVALID, dict(K=64)), (INVALID, dict(K=-128)), (MISALIGNED, dict(a=ODD)),
        (MISALIGNED, dict(sfa=ODD)), (MISALIGNED, dict(b=ODD)), (MISALIGNED, dict(sfb=ODD)), (MISALIGNED, dict(d=ODD)), (UNSUPPORTED, dict(M=BIG)),
        (UNSUPPORTED, dict(N=2 ** 31 - 16)), (UNSUPPORTED, dict(K=2 ** 31 - 128)), (OK, dict(M=0)), (OK, dict(M=0, a=None, d=None))]


@pytest.mark.parametrize("status, over", GEMM + [(MISALIGNED, dict(c=ODD))])
def test_gemm(L, status, over):
    assert gemm(L, **over) == status


@pytest.mark.parametrize("call", [masked, contiguous])
@pytest.mark.parametrize("status, over", GEMM + [(INVALID, dict(G=0)), (INVALID, dict(G=-3)), (INVALID, dict(counts=None)), (MISALIGNED, dict(counts=P(0x10002)))])
def test_grouped_gemm(L, call, status, over):
    assert call(L, **over) == status
