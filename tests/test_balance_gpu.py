"""dg_moe_balance_loss and its gradient against the FP64 oracle. Counts and live rows have to be equal.

A score's exponent x - top is at most 2^6 here and rounds to 2^-23 of itself in two operations, 2^-17 relative in the
score; the approximate 2^v, its reciprocal and the row's sum add a few 2^-22: p within 2^-16. Sums over rows are FP32: T
additions of values of one sign, in chains of at most T / 32 + 200, 2^-24 of the sum each. The gradient's difference
f - mean cancels: its error is 2^-15 of p (f + mean), the rounding to its type comes on top."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.four_bit as F

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    L.dg_get_device_status()
    return L


def make(T, E, dtype, seed, masked=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 2 * torch.randn(T, E, device="cuda", generator=g)
    if masked and T > 4:
        x[torch.rand(T, E, device="cuda", generator=g) < 0.2] = -float("inf")
        x[1] = -float("inf")                         # a row that is not live
        x[T // 2, ::2] = float("nan")
        x[2] = torch.finfo(dtype).min                # a row of the type's lowest value: all the same
        x[3, ::3] = torch.finfo(dtype).min
    return x.to(dtype)


def ids_of(x, k, seed):
    """Distinct experts of each row, some slots empty."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.argsort(torch.rand(x.shape, device="cuda", generator=g), -1)[:, :k].int()
    return torch.where(torch.rand(ids.shape, device="cuda", generator=g) < 0.1, -1, ids).contiguous()


def loss_of(L, x, ids, scoring, coef):
    E = x.shape[1]
    out = (torch.full((E,), -7, dtype=torch.int32, device="cuda"), torch.full((1,), -7, dtype=torch.int32, device="cuda"),
           torch.full((E,), float("nan"), device="cuda"), torch.full((1,), float("nan"), device="cuda"))
    assert L.dg_moe_balance_loss(x, ids, *out, scoring=scoring, coef=coef) is out[3]
    return out


def np64(t):
    return t.double().cpu().numpy()


def check_loss(x, ids, got, scoring, coef):
    loss, counts, live, mean = F.balance_loss(np64(x), ids.cpu().numpy(), scoring, coef)
    rel = 2.0 ** -16 + (len(x) / 32 + 200) * 2.0 ** -24
    assert (got[0].cpu().numpy() == counts).all() and int(got[1]) == live
    assert (np.abs(np64(got[2]) - mean) <= rel * mean + 2.0 ** -126).all()
    assert abs(float(got[3]) - loss) <= 2 * rel * abs(loss)


def check_gradient(x, counts, live, dloss, base, got, scoring, coef):
    x64 = np64(x)
    want = F.balance_loss_backward(x64, counts, live, dloss, scoring, coef)
    p, f = F.probabilities(x64, scoring), np.maximum(counts, 0) / max(np.maximum(counts, 0).sum(), 1)
    room = 2.0 ** -15 * abs(dloss * coef) * x.shape[1] / max(live, 1) * p * (f + (p @ f)[:, None])
    if base is not None:
        want = want + np64(base)
    assert (np.abs(np64(got) - want) <= room + 1.01 * HALF[x.dtype] * np.abs(want) + 2.0 ** -126).all()


SHAPES = [(1, 1, 1), (1, 256, 8), (5, 7, 7), (33, 31, 2), (40, 60, 4), (130, 100, 6), (17, 256, 16), (70, 33, 32), (8, 512, 32), (11, 1000, 12), (12, 1024, 1),
          (8, 1000, 2), (20, 1023, 5), (300, 33, 3), (128, 64, 2), (129, 61, 2), (3000, 64, 8), (5000, 256, 4)]


@pytest.mark.parametrize("T, E, k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_loss_and_gradient(lib, T, E, k, dtype, scoring):
    x = make(T, E, dtype, T + E + k)
    ids = ids_of(x, k, T)
    got = loss_of(lib, x, ids, scoring, 0.02)
    check_loss(x, ids, got, scoring, 0.02)
    dloss = torch.tensor([1.25], device="cuda")
    base = (torch.randn(T, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) / T).to(dtype)
    counts, live = got[0].cpu().numpy().astype(np.float64), int(got[1])
    for b in (None, base):
        dx = torch.full_like(x, float("nan"))
        assert lib.dg_moe_balance_loss_backward(x, got[0], got[1], dloss, dx, base=b, scoring=scoring, coef=0.02) is dx
        check_gradient(x, counts, live, 1.25, b, dx, scoring, 0.02)
    kept = base.clone()
    lib.dg_moe_balance_loss_backward(x, got[0], got[1], dloss, base, base=base, scoring=scoring, coef=0.02)     # in place
    assert torch.equal(base.view(torch.int16 if dtype == BF16 else torch.int32), dx.view(torch.int16 if dtype == BF16 else torch.int32))
    # an expert that is masked keeps the base's bits
    masked = ~(x > -float("inf"))
    assert torch.equal(base[masked], kept[masked])
    assert lib.dg_get_device_status() == 0


def test_gradient_by_differences(lib):
    # the loss at x + h d and x - h d, from the oracle, against <gradient, d>
    x = make(40, 24, F32, 5, masked=False)
    ids = ids_of(x, 3, 5)
    for scoring in ("softmax", "sigmoid"):
        got = loss_of(lib, x, ids, scoring, 1.0)
        dx = torch.empty_like(x)
        lib.dg_moe_balance_loss_backward(x, got[0], got[1], torch.ones(1, device="cuda"), dx, scoring=scoring)
        d, h = np.random.default_rng(6).normal(size=x.shape), 1e-5
        up, down = (F.balance_loss(np64(x) + s * h * d, ids.cpu().numpy(), scoring)[0] for s in (1, -1))
        # the difference's own error is h^2 of the third derivative (under 1) and 2^-52 of the loss over h
        assert abs((up - down) / (2 * h) - (np64(dx) * d).sum()) <= 2.0 ** -15 * np.abs(np64(dx) * d).sum() + 1e-9


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_rows(lib, dtype):
    store = make(90, 140, dtype, 7)
    x = store[4:84:5, 3:131]
    ids = ids_of(x, 4, 7)
    got = loss_of(lib, x, ids, "softmax", 1.0)
    check_loss(x, ids, got, "softmax", 1.0)
    same = loss_of(lib, x.contiguous(), ids, "softmax", 1.0)
    dx, dsame = torch.empty(16, 128, device="cuda", dtype=dtype), torch.empty(16, 128, device="cuda", dtype=dtype)
    one = torch.ones(1, device="cuda")
    lib.dg_moe_balance_loss_backward(x, got[0], got[1], one, dx)
    lib.dg_moe_balance_loss_backward(x.contiguous(), same[0], same[1], one, dsame)
    check_gradient(x, got[0].cpu().numpy().astype(np.float64), int(got[1]), 1.0, None, dx, "softmax", 1.0)
    check_gradient(x, got[0].cpu().numpy().astype(np.float64), int(got[1]), 1.0, None, dsame, "softmax", 1.0)


def test_no_rows(lib):
    x = torch.empty(0, 16, device="cuda")
    got = loss_of(lib, x, torch.empty(0, 2, dtype=torch.int32, device="cuda"), "softmax", 1.0)
    assert all((t == 0).all() for t in got)
    dx = torch.empty(0, 16, device="cuda")
    assert lib.dg_moe_balance_loss_backward(x, got[0], got[1], torch.ones(1, device="cuda"), dx) is dx


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_rows_that_are_not_live(lib, scoring):
    x = torch.full((50, 12), -float("inf"), device="cuda")
    ids = torch.full((50, 2), -1, dtype=torch.int32, device="cuda")
    got = loss_of(lib, x, ids, scoring, 1.0)
    assert all((t == 0).all() for t in got)
    dx = torch.full_like(x, 5.0)
    lib.dg_moe_balance_loss_backward(x, got[0], got[1], torch.ones(1, device="cuda"), dx, scoring=scoring)
    assert (dx == 0).all()


def test_small_sigmoids(lib):
    x = torch.full((8, 40), -300.0, device="cuda") + torch.arange(40, device="cuda") % 3
    ids = ids_of(x, 2, 8)
    check_loss(x, ids, loss_of(lib, x, ids, "sigmoid", 1.0), "sigmoid", 1.0)


def test_ids_out_of_range(lib):
    x = make(20, 16, F32, 9)
    ids = ids_of(x, 2, 9)
    want = ids.clone()
    ids[3, 0], ids[4, 1] = 16, -2
    want[3, 0], want[4, 1] = -1, -1
    got = loss_of(lib, x, ids, "softmax", 1.0)
    assert lib.dg_get_device_status() == 6
    check_loss(x, want, got, "softmax", 1.0)


def test_counts_of_other_batches(lib):
    # counts and live rows summed over batches, as data-parallel ranks do; a negative count is 0
    x = make(60, 32, F32, 10)
    counts = torch.arange(32, dtype=torch.int32, device="cuda") * 10 ** 7 - 5
    dx = torch.empty_like(x)
    lib.dg_moe_balance_loss_backward(x, counts, torch.tensor([1000], dtype=torch.int32, device="cuda"), torch.tensor([2.0], device="cuda"), dx)
    check_gradient(x, np.maximum(counts.cpu().numpy(), 0).astype(np.float64), 1000, 2.0, None, dx, "softmax", 1.0)


def test_the_same_bits_twice_and_in_a_graph(lib):
    x = make(4000, 256, F32, 11)
    ids = ids_of(x, 8, 11)
    first = loss_of(lib, x, ids, "softmax", 1.0)
    again = loss_of(lib, x, ids, "softmax", 1.0)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dx = torch.empty_like(x)
    one = torch.ones(1, device="cuda")
    with torch.cuda.stream(s):
        out = loss_of(lib, x, ids, "softmax", 1.0)
        lib.dg_moe_balance_loss_backward(x, out[0], out[1], one, dx)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            lib.dg_moe_balance_loss(x, ids, *out)
            lib.dg_moe_balance_loss_backward(x, out[0], out[1], one, dx)
        eager = dx.clone()
        for _ in range(2):
            for t in out + (dx,):
                t.zero_()
            g.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first, out)) and torch.equal(dx, eager)
        # new inputs in the same memory
        x.copy_(make(4000, 256, F32, 12))
        g.replay()
        s.synchronize()
    check_loss(x, ids, out, "softmax", 1.0)


@pytest.mark.parametrize("sms", [1, 2, 7])
def test_on_few_sms(lib, sms):
    # a block that is alone with all rows, and blocks that take their rows in many rounds
    for T, E, dtype, scoring in ((2000, 60, BF16, "sigmoid"), (700, 512, F32, "softmax")):
        x = make(T, E, dtype, 13)
        ids = ids_of(x, 6, 13)
        dx = torch.empty_like(x)
        try:
            lib.dg_set_num_sms(sms)
            got = loss_of(lib, x, ids, scoring, 0.5)
            lib.dg_moe_balance_loss_backward(x, got[0], got[1], torch.ones(1, device="cuda"), dx, scoring=scoring, coef=0.5)
        finally:
            lib.dg_set_num_sms(0)
        check_loss(x, ids, got, scoring, 0.5)
        check_gradient(x, got[0].cpu().numpy().astype(np.float64), int(got[1]), 1.0, None, dx, scoring, 0.5)


def test_two_streams_at_once(lib):
    sets = []
    for seed, T, E in ((14, 4000, 256), (15, 3500, 60)):
        x = make(T, E, F32, seed)
        ids = ids_of(x, 4, seed)
        sets.append((x, ids, loss_of(lib, x, ids, "softmax", 1.0), torch.cuda.Stream()))
    torch.cuda.synchronize()
    runs = []
    for _ in range(20):
        for x, ids, alone, s in sets:
            with torch.cuda.stream(s):
                runs.append((alone, loss_of(lib, x, ids, "softmax", 1.0)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for alone, got in runs for a, b in zip(alone, got))
