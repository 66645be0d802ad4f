"""dg_add_rms_norm and its gradient against the FP64 oracle.

Tolerances, from the arithmetic (u = 2^-24): a row's sum of squares is a chain of at most 64 FP32
additions per thread and a tree, so rstd is within 2^-18 of itself; y adds two roundings. A stored BF16
value is within 2^-8 of the FP32 one, a stored E4M3 code within half of its step: 2^-4 of the value, or
2^-10 of the scale among subnormals. The scale's code may differ from the exact one only where max|y|
lies within the FP32 error of 448 times a power of two."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
import oracle.layers as OL
import workloads as W

pytestmark = pytest.mark.gpu

F32_REL = 2.0 ** -17
BF16_REL = 2.0 ** -8


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    return L


def f64(t):
    return t.double().cpu().numpy()


def make(T, H, residual, weight, seed, with_residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    r = (3 * torch.randn(T, H, device="cuda", generator=g)).to(residual) if with_residual else None
    w = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(weight)
    return x, r, w


def outputs(L, T, H, dtype, q=True):
    o = {"residual_out": torch.full((T, H), float("nan"), dtype=dtype, device="cuda"),
         "y": torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda"),
         "rstd": torch.full((T,), float("nan"), device="cuda")}
    if q:
        o["q"] = torch.full((T, H), 0x7F, dtype=torch.uint8, device="cuda")
        o["sf"] = torch.full(L.sf_shape(T, H), -1, dtype=torch.int32, device="cuda")
    return o


def check(L, x, r, w, eps, o):
    T, H = x.shape
    s, rstd, y = OL.add_rms_norm(f64(x), None if r is None else f64(r), f64(w), eps)
    with np.errstate(invalid="ignore"):
        rel = BF16_REL if o["residual_out"].dtype == torch.bfloat16 else 2.0 ** -24
        assert (np.abs(f64(o["residual_out"]) - s) <= 1.001 * rel * np.abs(s)).all()
        assert (np.abs(f64(o["rstd"]) - rstd) <= F32_REL * rstd).all()
        assert (np.abs(f64(o["y"]) - y) <= (BF16_REL + F32_REL) * np.abs(y) + 2.0 ** -134).all()
    if "q" not in o:
        return
    words = o["sf"].cpu().numpy()
    codes = O.unpack_sf(words, T, H // 128).astype(np.int64)
    want = OL.group_scale_codes(y)
    amax = np.abs(y).reshape(T, H // 128, 128).max(-1)
    edge = np.ldexp(448.0, np.minimum(codes, want) - 127)
    assert ((codes == want) | ((np.abs(codes - want) == 1) & (np.abs(amax - edge) <= F32_REL * edge))).all()
    scale = np.repeat(np.ldexp(1.0, codes - 127), 128, 1)
    got = O.decode_e4m3(o["q"].cpu().numpy()) * scale
    assert (np.abs(got - y) <= 1.001 * np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * scale) + F32_REL * np.abs(y)).all()
    # padding rows and bytes are zero
    b = np.ascontiguousarray(words).view(np.uint8).reshape(words.shape[0], -1, 4)
    assert not b[:, T:].any()
    flat = b.transpose(1, 0, 2).reshape(b.shape[1], -1)
    assert not flat[:, H // 128:].any()


@pytest.mark.parametrize("T, H", [(1, 128), (2, 7168), (3, 640), (5, 2176), (130, 2048), (33, 16384), (9, 4096)])
@pytest.mark.parametrize("residual, weight", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                              (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_all_outputs(lib, T, H, residual, weight):
    x, r, w = make(T, H, residual, weight, seed=T * H)
    o = outputs(lib, T, H, residual)
    lib.dg_add_rms_norm(x, r, w, 1e-6, **o)
    check(lib, x, r, w, 1e-6, o)
    assert lib.dg_get_device_status() == 0


@pytest.mark.parametrize("H", [8, 64, 136, 1000, 5000])
def test_widths_without_scales(lib, H):
    x, r, w = make(7, H, torch.bfloat16, torch.bfloat16, seed=H)
    o = outputs(lib, 7, H, torch.bfloat16, q=False)
    lib.dg_add_rms_norm(x, r, w, 1e-5, **o)
    check(lib, x, r, w, 1e-5, o)


def test_each_output_alone_and_no_residual(lib):
    T, H = 6, 512
    x, r, w = make(T, H, torch.bfloat16, torch.bfloat16, seed=4)
    full = outputs(lib, T, H, torch.bfloat16)
    lib.dg_add_rms_norm(x, r, w, 1e-6, **full)
    for names in (("y",), ("residual_out",), ("q", "sf"), ("residual_out", "rstd")):
        o = {k: v for k, v in outputs(lib, T, H, torch.bfloat16).items() if k in names}
        lib.dg_add_rms_norm(x, r, w, 1e-6, **o)
        for k, v in o.items():
            assert torch.equal(v, full[k]), k
    o = outputs(lib, T, H, torch.bfloat16)
    lib.dg_add_rms_norm(x, None, w, 1e-6, **o)
    check(lib, x, None, w, 1e-6, o)
    assert torch.equal(o["residual_out"], x)


def test_strided_rows_and_in_place(lib):
    T, H = 5, 384
    x, r, w = make(T, H, torch.float32, torch.bfloat16, seed=5)
    want = outputs(lib, T, H, torch.float32)
    lib.dg_add_rms_norm(x, r, w, 1e-6, **want)
    xs = torch.full((T, H + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    rs = torch.full((T, 2 * H), float("nan"), device="cuda")
    xs[:, :H], rs[:, :H] = x, r
    o = outputs(lib, T, H, torch.float32)
    o["residual_out"] = rs[:, :H]                    # in place, strided
    lib.dg_add_rms_norm(xs[:, :H], rs[:, :H], w, 1e-6, **o)
    for k in want:
        assert torch.equal(o[k], want[k]), k
    assert rs[:, H:].isnan().all() and xs[:, H:].isnan().all()
    y = x.clone()
    lib.dg_add_rms_norm(y, r, w, 1e-6, y=y)          # y over x
    assert torch.equal(y, want["y"])


def test_zero_rows_extremes_and_what_is_not_finite(lib):
    T, H = 5, 256
    x = torch.randn(T, H, device="cuda").bfloat16()
    x[0] = 0
    x[1] *= 2.0 ** 60                                 # squares reach 2^120 each
    x[2] *= 2.0 ** -70                                # squares underflow: rstd is eps's
    x[3, 5] = float("nan")
    w = torch.ones(H, device="cuda")
    w[7] = float("inf")
    w[128:] = 2.0 ** -100                             # scales far below 1
    o = outputs(lib, T, H, torch.bfloat16)
    lib.dg_add_rms_norm(x, None, w, 1e-6, **o)
    y, q = o["y"].float(), o["q"]
    codes = O.unpack_sf(o["sf"].cpu().numpy(), T, 2)
    assert o["rstd"][0].item() == pytest.approx(1e3, rel=1e-6)
    assert (y[0, :7] == 0).all() and y[0, 7].isnan()  # 0 * inf
    assert y[1, 7].isinf() and (q[1, 7] & 0x7F) == 0x7F
    assert codes[0].tolist() == [127, 127]
    keep = [i for i in range(128) if i != 7]
    y64 = f64(x)[1] / np.sqrt(np.mean(f64(x)[1] ** 2) + 1e-6)
    assert codes[1, 0] == OL.group_scale_codes(np.where(np.arange(128) == 7, 0, y64[:128])[None])[0, 0]
    got = O.decode_e4m3(q[1].cpu().numpy())[keep] * 2.0 ** (int(codes[1, 0]) - 127)
    assert (np.abs(got - y64[keep]) <= 2.0 ** -4 * np.abs(y64[keep]) * 1.01 + 2.0 ** -10 * 2.0 ** (int(codes[1, 0]) - 127)).all()
    assert abs(int(codes[1, 1]) - int(codes[4, 1])) <= 2 and codes[1, 1] < 30      # the 2^-100 half
    assert codes[2, 0] >= 1 and o["rstd"][2].item() == pytest.approx(1e3, rel=1e-6)
    assert y[3].isnan().all() and ((q[3] & 0x7F) == 0x7F).all() and codes[3].tolist() == [127, 127]


def test_rows_past_four_gib(lib):
    # 2^31 elements and more: the last rows must be those of a small call
    H = 7168
    T = (1 << 31) // H + 70
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x[:-64] = 1
    x[-64:] = torch.randn(64, H, device="cuda").bfloat16()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    sf = torch.empty(lib.sf_shape(T, H), dtype=torch.int32, device="cuda")
    lib.dg_add_rms_norm(x, None, w, 0.0, q=q, sf=sf, residual_out=x)
    qs = torch.empty(64, H, dtype=torch.float8_e4m3fn, device="cuda")
    sfs = torch.empty(lib.sf_shape(64, H), dtype=torch.int32, device="cuda")
    lib.dg_add_rms_norm(x[-64:], None, w, 0.0, q=qs, sf=sfs)
    assert torch.equal(q[-64:].view(torch.uint8), qs.view(torch.uint8))
    assert torch.equal(sf[:, T - 64:T], sfs)


@pytest.mark.parametrize("T, H", [(1, 8), (3, 128), (301, 2048), (640, 1000), (37, 7168), (5, 16384), (2, 4096), (331, 5120)])
@pytest.mark.parametrize("residual, weight", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                              (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_gradient(lib, T, H, residual, weight):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    s, ds = [(k * torch.randn(T, H, device="cuda", generator=g)).to(residual) for k in (3, 1)]
    dy = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    w = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(weight)
    rstd = (f := s.float().square().mean(-1) + 1e-6).rsqrt()
    dx = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dr = torch.full((T, H), float("nan"), dtype=residual, device="cuda")
    dw = torch.full((H,), float("nan"), device="cuda")
    lib.dg_add_rms_norm_backward(dy, s, w, rstd, ds, dx, dr, dw)
    want, want_w = OL.add_rms_norm_backward(f64(dy), f64(s), f64(w), f64(rstd), f64(ds))
    xhat = f64(s) * f64(rstd)[:, None]
    gy = f64(dy) * f64(w)
    # the mean is a sum of at most 64 + log terms per thread; every other step rounds once or twice
    tol = F32_REL * (f64(rstd)[:, None] * (np.abs(gy) + np.abs(xhat) * np.mean(np.abs(gy * xhat), -1, keepdims=True)) + np.abs(f64(ds)))
    assert (np.abs(f64(dx) - want) <= BF16_REL * np.abs(want) + 2 * tol).all()
    rel = BF16_REL if residual == torch.bfloat16 else 2.0 ** -24
    assert (np.abs(f64(dr) - want) <= rel * np.abs(want) + 2 * tol).all()
    # dw: chains of at most T / 2 + 300 / 8 FP32 additions
    assert (np.abs(f64(dw) - want_w) <= (T + 64) * 2.0 ** -24 * np.abs(f64(dy) * xhat).sum(0)).all()


def test_gradient_variants(lib):
    T, H = 50, 640
    g = torch.Generator(device="cuda").manual_seed(9)
    s, ds = [torch.randn(T, H, device="cuda", generator=g) for _ in range(2)]
    dy = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    w = torch.randn(H, device="cuda", generator=g)
    rstd = s.square().mean(-1).rsqrt()
    run = lambda ds, dx, dr, dy=dy: [lib.dg_add_rms_norm_backward(dy, s, w, rstd, ds, dx, dr, dw), dw.clone()][1]  # noqa: E731
    dw = torch.empty(H, device="cuda")
    dx, dr = torch.empty_like(dy), torch.empty_like(s)
    first = run(ds, dx, dr)
    assert torch.equal(run(ds, None, dr.clone()), first) and torch.equal(run(ds, dx.clone(), None), first)   # same bits again
    dr0 = torch.empty_like(s)
    run(None, None, dr0)
    want, _ = OL.add_rms_norm_backward(f64(dy), f64(s), f64(w), f64(rstd), None)
    assert np.abs(f64(dr0) - want).max() <= 2.0 ** -16 * np.abs(want).max()
    inplace, dyc = ds.clone(), dy.clone()
    assert torch.equal(run(inplace, dyc, inplace, dy=dyc), first) and torch.equal(inplace, dr) and torch.equal(dyc, dx)
    empty = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    lib.dg_add_rms_norm_backward(empty, s[:0], w, rstd[:0], None, empty, None, dw)
    assert (dw == 0).all()


def test_gradient_matches_differences_of_the_forward(lib):
    # <d, v> against (f(s + t v) - f(s - t v)) / 2t with f = sum(dy * y) of the library's own FP32 rstd
    # and the definition's y in FP64: step 2^-7 on values of size 1, error O(t^2) = 2^-14 and rounding 2^-17 / t
    T, H = 4, 256
    g = torch.Generator(device="cuda").manual_seed(10)
    s, v, w = [torch.randn(*d, device="cuda", generator=g) for d in ((T, H), (T, H), (H,))]
    dy = torch.randn(T, H, device="cuda", generator=g).bfloat16()

    def rstd(z):
        r, o = torch.empty(T, device="cuda"), torch.empty_like(z)
        lib.dg_add_rms_norm(torch.zeros_like(dy), z, w, 1e-6, residual_out=o, rstd=r)
        assert torch.equal(o, z)
        return r

    def f(z):
        return (dy.double() * z.double() * rstd(z).double()[:, None] * w.double()).sum().item()

    t = 2.0 ** -7
    dr, dw = torch.empty_like(s), torch.empty(H, device="cuda")
    lib.dg_add_rms_norm_backward(dy, s, w, rstd(s), None, None, dr, dw)
    got, want = (dr.double() * v.double()).sum().item(), (f(s + t * v) - f(s - t * v)) / (2 * t)
    assert abs(got - want) <= 2e-3 * np.sqrt(T * H)


def test_streams_graph_and_pdl(lib):
    T, H = 40, 1024
    x, r, w = make(T, H, torch.bfloat16, torch.bfloat16, seed=11)
    want = outputs(lib, T, H, torch.bfloat16)
    lib.dg_add_rms_norm(x, r, w, 1e-6, **want)
    dwant, dww = torch.empty_like(x), torch.empty(H, device="cuda")
    lib.dg_add_rms_norm_backward(x, want["residual_out"], w, want["rstd"], r, dwant, None, dww)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, dx, dw = outputs(lib, T, H, torch.bfloat16), torch.empty_like(x), torch.empty(H, device="cuda")

    def both():
        lib.dg_add_rms_norm(x, r, w, 1e-6, **o, stream=s)
        lib.dg_add_rms_norm_backward(x, o["residual_out"], w, o["rstd"], r, dx, None, dw, stream=s)

    def same():
        torch.cuda.synchronize()
        ok = all(torch.equal(o[k], want[k]) for k in want) and torch.equal(dx, dwant) and torch.equal(dw, dww)
        for v in (*o.values(), dx, dw):
            v.zero_()
        torch.cuda.synchronize()
        return ok

    try:
        for pdl in (0, 1):
            lib.dg_set_pdl(pdl)
            both()
            assert same(), pdl
    finally:
        lib.dg_set_pdl(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for _ in range(2):
        graph.replay()
        assert same()
    lib.dg_set_num_sms(7)
    try:
        both()
        torch.cuda.synchronize()
        assert torch.equal(dx, dwant) and torch.allclose(dw, dww, rtol=0, atol=2.0 ** -18 * T * 3)
    finally:
        lib.dg_set_num_sms(0)


def test_output_feeds_the_gemm(lib):
    M, K, N = 70, 512, 256
    x, r, w = make(M, K, torch.bfloat16, torch.bfloat16, seed=12)
    o = outputs(lib, M, K, torch.bfloat16)
    lib.dg_add_rms_norm(x, r, w, 1e-6, **o)
    p = W.make_dense(M, N, K, seed=3)
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    b, sfb = torch.from_numpy(p.b).cuda(), torch.from_numpy(p.sfb).cuda()
    lib.dg_fp8_gemm_nt(o["q"], o["sf"], b, sfb, None, d)
    ref = O.fp8_gemm_nt(o["q"].cpu().numpy(), o["sf"].cpu().numpy(), p.b, p.sfb, None, M, N, K)
    assert O.parity_report(f64(d), ref)["ok"]


def test_binding_refuses(lib):
    x, r, w = make(4, 128, torch.bfloat16, torch.bfloat16, seed=13)
    y = torch.empty_like(x)
    q, sf = torch.empty(4, 128, dtype=torch.uint8, device="cuda"), torch.empty(1, 4, dtype=torch.int32, device="cuda")
    norm = lambda *a, **k: lib.dg_add_rms_norm(*a, **k)  # noqa: E731
    with pytest.raises(ValueError, match="bf16"):
        norm(x.float(), r, w, 1e-6, y=y)
    with pytest.raises(ValueError, match="shape"):
        norm(x, r[:3], w, 1e-6, y=y)
    with pytest.raises(ValueError, match="contiguous columns"):
        norm(x, r.t().contiguous().t(), w, 1e-6, y=y)
    with pytest.raises(ValueError, match="type"):
        norm(x, r, w, 1e-6, residual_out=r.float())
    with pytest.raises(ValueError, match="sf shape"):
        norm(x, r, w, 1e-6, q=q, sf=sf[:, :3].contiguous())
    with pytest.raises(ValueError, match="CUDA"):
        norm(x.cpu(), r, w, 1e-6, y=y)
    for bad in (dict(q=q), dict(sf=sf), dict()):
        with pytest.raises(lib.DGError, match="INVALID"):
            norm(x, r, w, 1e-6, **bad)
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(lib.DGError, match="INVALID"):
            norm(x, r, w, eps, y=y)
    odd = torch.empty(4, 132, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lib.DGError, match="MISALIGNED"):
        norm(odd[:, :128], r, w, 1e-6, y=y)          # rows 264 bytes apart
    with pytest.raises(lib.DGError, match="MISALIGNED"):
        norm(torch.empty(4 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 128), r, w, 1e-6, y=y)
    big = torch.empty(1, 16392, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lib.DGError, match="UNSUPPORTED"):
        norm(big, None, big[0], 1e-6, y=big.clone())
    dw = torch.empty(128, device="cuda")
    with pytest.raises(lib.DGError, match="INVALID"):
        lib.dg_add_rms_norm_backward(x, r, w, dw[:4], None, None, None, dw)
    with pytest.raises(ValueError, match="type"):
        lib.dg_add_rms_norm_backward(x, r, w, dw[:4], r.float(), y, None, dw)
