"""dg_moe_route and its gradient against the FP64 oracle. Ids have to be equal. Weights are FP32: the
argument x - max of the exponential rounds to 2^-24 of itself (at most 2^5 here: 2^-19 relative in the
exponential), the rest is a few roundings and a tree sum of at most 1024 terms: 2^-17 of the value."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.layers as OL

pytestmark = pytest.mark.gpu

REL = 2.0 ** -17


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    return L


def make(T, E, dtype, seed, masked=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 2 * torch.randn(T, E, device="cuda", generator=g)
    if masked and T > 2:
        x[torch.rand(T, E, device="cuda", generator=g) < 0.2] = -float("inf")
        x[1] = -float("inf")
        x[T // 2, ::2] = float("nan")
        x[0] = x[0].round()                          # ties, both zeros among them
        x[0, ::3] = -0.0
    return x.to(dtype)


def route(L, x, k, scoring, renorm, scale=1.0):
    ids = torch.full((len(x), k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((len(x), k), float("nan"), device="cuda")
    L.dg_moe_route(x, ids, w, scoring, renorm, scale)
    return ids, w


SHAPES = [(1, 1, 1), (1, 256, 8), (5, 7, 7), (33, 31, 2), (9, 33, 32), (40, 60, 4), (130, 100, 6), (17, 256, 16), (8, 512, 32), (11, 1000, 12),
          (12, 1024, 1)]


@pytest.mark.parametrize("T, E, k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring, renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_and_gradient(lib, T, E, k, dtype, scoring, renorm):
    x = make(T, E, dtype, seed=T + E + k)
    ids, w = route(lib, x, k, scoring, renorm, 2.5)
    x64 = x.double().cpu().numpy()
    want_ids, want = OL.moe_route(x64, k, scoring, renorm, 2.5)
    assert (ids.cpu().numpy() == want_ids).all()
    assert (np.abs(w.double().cpu().numpy() - want) <= REL * np.abs(want)).all()

    dw = torch.randn(T, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    dw[ids < 0] = float("nan")                       # not read as values
    dx = torch.full_like(x, float("nan"))
    lib.dg_moe_route_backward(x, ids, dw, dx, scoring, renorm, 2.5)
    d64 = torch.nan_to_num(dw, nan=0.0).double().cpu().numpy()
    grad = OL.moe_route_backward(x64, want_ids, d64, scoring, renorm, 2.5)
    # every term is at most |scale d| (p / sum p <= 1) times a few roundings; BF16 rounds once more
    tol = REL * 2.5 * np.abs(d64).sum(-1, keepdims=True) + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * np.abs(grad)
    if k:
        assert (np.abs(dx.double().cpu().numpy() - grad) <= tol).all()
    assert lib.dg_get_device_status() == 0


@pytest.mark.parametrize("T, E, k", [(8193, 64, 8), (8192, 40, 1), (9001, 250, 5), (8200, 256, 8), (8193, 100, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring, renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_two_rows_a_warp(lib, T, E, k, dtype, scoring, renorm):
    # two rows a warp, among them rows of ties, which have many candidates, and rows with few or no experts left;
    # the same bits as in calls of fewer rows
    x = make(T, E, dtype, seed=T + E + k)
    x[5::7] = x[5::7].round()
    x[100:300:3] = 1.0
    x[301:320] = -float("inf")
    x[310:315, E // 2] = -3.0
    x[T - 1] = float("nan")
    x[T - 2, : E // 2] = 2.0
    ids, w = route(lib, x, k, scoring, renorm, 0.5)
    few = [route(lib, x[i:i + 3000], k, scoring, renorm, 0.5) for i in range(0, T, 3000)]
    assert torch.equal(ids, torch.cat([f[0] for f in few])) and torch.equal(w, torch.cat([f[1] for f in few]))
    some = np.r_[0:700, T - 300:T]
    want_ids, want = OL.moe_route(x[torch.from_numpy(some).cuda()].double().cpu().numpy(), k, scoring, renorm, 0.5)
    assert (ids.cpu().numpy()[some] == want_ids).all()
    assert (np.abs(w.double().cpu().numpy()[some] - want) <= REL * np.abs(want)).all()


def test_infinite_and_extreme_logits(lib):
    inf = float("inf")
    x = torch.tensor([[inf, 0.0, 1.0], [-200.0, -300.0, -inf], [3e38, -3e38, 0.0], [float("nan")] * 3], device="cuda")
    ids, w = route(lib, x, 2, "softmax", True)
    assert ids.tolist() == [[0, 2], [0, 1], [0, 2], [-1, -1]]
    assert w[0].isnan().all() and w[1].tolist() == pytest.approx([1.0, np.exp(-100.0)], abs=2.0 ** -149) and w[2].tolist() == [1.0, 0.0] and w[3].tolist() == [0.0, 0.0]
    ids, w = route(lib, x, 2, "sigmoid", True)       # both scores of row 1 underflow to 0
    assert w[0].tolist() == pytest.approx([1 / (1 + 1 / (1 + np.exp(-1.0))), 1 / (1 + (1 + np.exp(-1.0)))])
    assert w[1].tolist() == [0.0, 0.0] and w[2].tolist() == pytest.approx([2 / 3, 1 / 3])
    dx = torch.empty_like(x)
    lib.dg_moe_route_backward(x, ids, torch.ones(4, 2, device="cuda"), dx, "sigmoid", True)
    assert (dx[1] == 0).all() and (dx[3] == 0).all()


def test_strided_logits_stream_graph(lib):
    T, E, k = 37, 96, 5
    x = make(T, E, torch.bfloat16, seed=3)
    ids, w = route(lib, x, k, "softmax", True)
    wide = torch.full((T, 131), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:99] = x                                # rows 262 bytes apart, at an odd offset
    s = torch.cuda.Stream()
    ids2, w2, dx2 = torch.zeros_like(ids), torch.zeros_like(w), torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()

    def both():
        lib.dg_moe_route(wide[:, 3:99], ids2, w2, stream=s)
        lib.dg_moe_route_backward(wide[:, 3:99], ids2, w2, dx2, stream=s)

    both()
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    first = dx2.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for v in (ids2, w2, dx2):
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(dx2, first)


def test_many_rows(lib):
    # more than 2^31 logits: the last rows are those of a small call
    E, k = 1024, 4
    T = (1 << 31) // E + 9
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    x[-16:] = torch.randn(16, E, device="cuda").bfloat16()
    ids, w = route(lib, x, k, "softmax", False)
    small_ids, small_w = route(lib, x[-16:].clone(), k, "softmax", False)
    assert torch.equal(ids[-16:], small_ids) and torch.equal(w[-16:], small_w)
    assert (ids[:-16] == torch.arange(k, device="cuda")).all()


def test_bad_ids_are_reported(lib):
    x = make(4, 8, torch.float32, seed=4, masked=False)
    ids = torch.tensor([[0, 1], [8, 2], [-2, 3], [4, -1]], dtype=torch.int32, device="cuda")
    dx = torch.empty_like(x)
    lib.dg_moe_route_backward(x, ids, torch.ones(4, 2, device="cuda"), dx, "sigmoid", False)
    assert lib.dg_get_device_status() == 6 and lib.dg_get_device_status() == 0
    want = OL.moe_route_backward(x.double().cpu().numpy(), np.array([[0, 1], [-1, 2], [-1, 3], [4, -1]]), np.ones((4, 2)), "sigmoid", False)
    assert np.abs(dx.double().cpu().numpy() - want).max() <= REL


def test_binding_refuses(lib):
    x = make(3, 8, torch.float32, seed=5, masked=False)
    ids, w = torch.empty(3, 2, dtype=torch.int32, device="cuda"), torch.empty(3, 2, device="cuda")
    for bad in (lambda: lib.dg_moe_route(x.half(), ids, w), lambda: lib.dg_moe_route(x, ids.long(), w),
                lambda: lib.dg_moe_route(x, ids, w[:2]), lambda: lib.dg_moe_route(x, ids, w, scoring="relu"),
                lambda: lib.dg_moe_route(x.t().contiguous().t(), ids, w), lambda: lib.dg_moe_route(x[0], ids, w),
                lambda: lib.dg_moe_route_backward(x, ids, w, x.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lib.DGError, match="INVALID"):
        lib.dg_moe_route(x, torch.empty(3, 9, dtype=torch.int32, device="cuda"), torch.empty(3, 9, device="cuda"))
    with pytest.raises(lib.DGError, match="INVALID"):
        lib.dg_moe_route(x, ids, w, scale=float("nan"))
    with pytest.raises(lib.DGError, match="UNSUPPORTED"):
        lib.dg_moe_route(torch.zeros(3, 1025, device="cuda"), ids, w)
    with pytest.raises(lib.DGError, match="UNSUPPORTED"):
        lib.dg_moe_route(torch.zeros(3, 64, device="cuda"), torch.empty(3, 33, dtype=torch.int32, device="cuda"), torch.empty(3, 33, device="cuda"))
