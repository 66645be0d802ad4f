"""Arguments that the operators around the GEMMs refuse before they touch the device (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest

P = ctypes.c_void_p
X = P(0x10000)           # never dereferenced: validation fails first
ODD = P(0x10008)
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from fp8_gemm_nt_gb300 import build
    build.build()
    import fp8_gemm_nt_gb300 as pkg
    pkg.load_library()
    return pkg


def norm(L, x=X, residual=X, weight=X, out=X, y=X, q=X, sf=X, rstd=X, T=4, H=256, ldx=256, ldr=256, ldo=256, rt=0, wt=0, eps=1e-6):
    d = L._NormDesc(T, H, ldx, ldr, ldo, rt, wt, eps)
    return L.load_library().dg_add_rms_norm(x, residual, weight, out, y, q, sf, rstd, ctypes.byref(d), None)


@pytest.mark.parametrize("status, over", [
    (INVALID, dict(x=None)), (INVALID, dict(weight=None)), (INVALID, dict(T=-1)), (INVALID, dict(H=0)), (INVALID, dict(H=260)),
    (INVALID, dict(H=264, ldx=264, ldr=264, ldo=264)), (INVALID, dict(q=None)), (INVALID, dict(sf=None)), (INVALID, dict(rt=2)), (INVALID, dict(wt=-1)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(ldx=128)), (INVALID, dict(ldr=248)), (INVALID, dict(ldo=0)),
    (INVALID, dict(out=None, y=None, q=None, sf=None)), (UNSUPPORTED, dict(H=16512, ldx=16512, ldr=16512, ldo=16512)),
    (MISALIGNED, dict(x=ODD)), (MISALIGNED, dict(sf=ODD)), (MISALIGNED, dict(ldx=260)), (MISALIGNED, dict(rt=1, ldr=258)), (MISALIGNED, dict(rstd=P(0x10002))),
    (OK, dict(T=0, x=None, weight=None, q=None, sf=None)), (OK, dict(T=0))])
def test_norm(L, status, over):
    assert norm(L, **over) == status


def test_norm_without_sizes(L):
    assert L.load_library().dg_add_rms_norm(X, X, X, X, X, X, X, X, None, None) == INVALID


def grad(L, dy=X, s=X, weight=X, rstd=X, ds=X, dx=X, dr=X, dw=X, T=4, H=256, rt=0, wt=0):
    return L.load_library().dg_add_rms_norm_backward(dy, s, weight, rstd, ds, dx, dr, dw, T, H, rt, wt, None)


@pytest.mark.parametrize("status, over", [
    (INVALID, dict(dy=None)), (INVALID, dict(s=None)), (INVALID, dict(weight=None)), (INVALID, dict(rstd=None)), (INVALID, dict(dw=None)),
    (INVALID, dict(dx=None, dr=None)), (INVALID, dict(T=-2)), (INVALID, dict(H=4)), (INVALID, dict(rt=5)), (UNSUPPORTED, dict(H=16392)),
    (MISALIGNED, dict(dy=ODD)), (MISALIGNED, dict(ds=ODD)), (MISALIGNED, dict(dw=ODD))])
def test_norm_gradient(L, status, over):
    assert grad(L, **over) == status


def route(L, logits=X, ids=X, w=X, T=4, E=16, k=2, ld=16, lt=1, scoring=0, renorm=1, scale=1.0):
    d = L._RouteDesc(T, E, k, ld, lt, scoring, renorm, scale)
    lib = L.load_library()
    return lib.dg_moe_route(logits, ids, w, ctypes.byref(d), None), lib.dg_moe_route_backward(logits, ids, w, X, ctypes.byref(d), None)


@pytest.mark.parametrize("status, over", [
    (INVALID, dict(logits=None)), (INVALID, dict(ids=None)), (INVALID, dict(w=None)), (INVALID, dict(T=-1)), (INVALID, dict(E=0)), (INVALID, dict(k=0)),
    (INVALID, dict(k=17)), (INVALID, dict(ld=15)), (INVALID, dict(lt=3)), (INVALID, dict(scoring=2)), (INVALID, dict(renorm=2)), (INVALID, dict(scale=float("inf"))),
    (UNSUPPORTED, dict(E=1025, ld=1025)), (UNSUPPORTED, dict(E=64, ld=64, k=33)), (MISALIGNED, dict(logits=P(0x10002))), (MISALIGNED, dict(ids=P(0x10002))),
    (MISALIGNED, dict(lt=0, logits=P(0x10001))), (OK, dict(T=0, logits=None, ids=None, w=None))])
def test_route(L, status, over):
    assert route(L, **over) == (status, status)


def test_route_without_sizes_or_output(L):
    lib = L.load_library()
    assert lib.dg_moe_route(X, X, X, None, None) == INVALID
    assert lib.dg_moe_route_backward(X, X, X, X, None, None) == INVALID
    d = L._RouteDesc(4, 16, 2, 16, 1, 0, 1, 1.0)
    assert lib.dg_moe_route_backward(X, X, X, None, ctypes.byref(d), None) == INVALID
    assert lib.dg_moe_route_backward(X, X, X, P(0x10002), ctypes.byref(d), None) == MISALIGNED


NAMES = ("x", "sfx", "w13", "sf13", "w2", "sf2", "ids", "weights", "c", "y")


@pytest.mark.parametrize("fn", ["dg_moe_fp8_few_tokens", "dg_moe_fp8_fp4_few_tokens"])
def test_few_tokens(L, fn):
    def call(T=4, k=2, E=8, H=256, I=128, **over):
        return getattr(L.load_library(), fn)(*[over.get(n, X) for n in NAMES], T, k, E, H, I, None)

    for n in NAMES:
        if n != "c":
            assert call(**{n: None}) == INVALID, n
        assert call(**{n: P(0x10002)}) == MISALIGNED, n
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(H=0), dict(I=-128), dict(H=200), dict(I=64)):
        assert call(**bad) == INVALID, bad
    for big in (dict(T=33), dict(k=17), dict(E=1025), dict(H=16512), dict(I=16512)):
        assert call(**big) == UNSUPPORTED, big
    assert call(T=0, **{n: None for n in NAMES}) == OK
