"""Every kernel of the FP4 x FP4 products, by the sizes of fp4_ways.py (which tests/test_fp4_ways.py holds to the kernels they
stand for), against the FP64 oracle; and what the kernel of CTA pairs has its own way with, at each width of its tiles in each
form: C that is D, scales over a wide range, at the ends and 255, places of K, addends that are not finite.

Exact cases and tolerances as in test_fp4_gemm_gpu.py: where FP32 holds every partial sum D has to be the one rounding of the
exact sum; otherwise each of the K / 64 instructions rounds a partial sum, by 2^-22 of the terms' magnitudes at most, and D
is rounded to 2^-8."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.four_bit as F
import workloads as W
from fp4_ways import CONTIGUOUS, DENSE, MASKED, PAIRS
from gpu_util import bf16_bits, dev, sentinel_like
from test_fp4_gemm_gpu import BF16, Operand, bits_of, check_exact, pair, rounded, spread, stacked

pytestmark = pytest.mark.gpu

EACH_PAIR = [(form, bn) for form in PAIRS for bn in PAIRS[form]]
SPECIAL = [(form, PAIRS[form][bn]) for form, bn in EACH_PAIR]


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    L.dg_get_device_status()
    return L


class Product:
    """One product of a form: its operands (A in one piece, but for the masked form), and the rows of D that go with each of B."""

    def __init__(self, form, size, seed, a_range=None, b_range=None):
        rng = np.random.default_rng(seed)
        self.form = form
        if form == "dense":
            (M, N, K), G = size, 1
        elif form == "contiguous":
            M, N, K, G = size
        else:
            G, M, N, K = size
        s = spread(K)
        a_range, b_range = a_range or (127, 127 + s // 2), b_range or (127, 127 + s - s // 2)
        self.a = [Operand(rng, M, K, *a_range) for _ in range(G if form == "masked" else 1)]
        self.b = [Operand(rng, N, K, *b_range) for _ in range(G)]
        self.M, self.N, self.K = M, N, K
        if form == "contiguous":
            # the experts' blocks of 128 rows, the last one of each not full; an expert without any
            assert M % 128 == 0
            cuts = np.sort(rng.integers(0, M // 128 + 1, G - 1))
            cuts[:1] = cuts[1:2]
            self.index = np.full(M, -1, np.int32)
            for e, (lo, hi) in enumerate(zip([0, *cuts], [*cuts, M // 128])):
                if hi > lo:
                    self.index[128 * lo:128 * hi - rng.integers(0, 128)] = e
            self.rows = [np.flatnonzero(self.index == e) for e in range(G)]
        elif form == "masked":
            self.counts = rng.integers(0, M + 1, G).astype(np.int32)
            self.counts[:2] = M, 0
            self.rows = [np.arange(c) for c in self.counts]
        else:
            self.rows = [np.arange(M)]

    def operand(self, g):
        return self.a[g if self.form == "masked" else 0]

    def repack(self):
        for o in (*self.a, *self.b):
            o.sf = W.pack_sf(o.exps)

    def call(self, L):
        """(the call with a stream, D)."""
        (da, dsa), (db, dsb) = stacked(self.a), stacked(self.b)
        if self.form == "masked":
            d, counts = sentinel_like((len(self.a), self.M, self.N)), dev(self.counts)
            return lambda s=None: L.dg_m_grouped_fp4_gemm_nt_masked(da, dsa, db, dsb, d, counts, stream=s), d
        d = sentinel_like((self.M, self.N))
        if self.form == "contiguous":
            index = dev(self.index)
            return lambda s=None: L.dg_m_grouped_fp4_gemm_nt_contiguous(da[0], dsa[0], db, dsb, d, index, stream=s), d
        return lambda s=None: L.dg_fp4_gemm_nt(da[0], dsa[0], db[0], dsb[0], None, d, stream=s), d

    def run(self, L):
        call, d = self.call(L)
        before = bf16_bits(d).copy()
        call()
        assert L.dg_get_device_status() == 0
        got = bf16_bits(d)
        # what the form does not compute is left as it was
        for g in range(len(got) if self.form == "masked" else 1):
            at = got[g] if self.form == "masked" else got
            was = before[g] if self.form == "masked" else before
            done = np.zeros(self.M, bool)
            for r in [self.rows[g]] if self.form == "masked" else self.rows:
                done[r] = True
            assert (at[~done] == was[~done]).all()
        return got

    def parts(self, got):
        """For each group with rows: (group, D's bits of its rows, values of A's rows, values of B)."""
        av = [F.values(o.packed, o.sf) for o in self.a]
        for g, r in enumerate(self.rows):
            if len(r):
                yield g, (got[g] if self.form == "masked" else got)[r], av[g if self.form == "masked" else 0][r], F.values(self.b[g].packed, self.b[g].sf)


def floats(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("size", [s for s, _ in DENSE])
@pytest.mark.parametrize("with_c", [False, True])
def test_dense(lib, size, with_c):
    check_exact(lib, *pair(sum(size), *size), with_c, seed=size[0])


@pytest.mark.parametrize("form, size", [("contiguous", s) for s, _ in CONTIGUOUS] + [("masked", s) for s, _ in MASKED])
def test_grouped(lib, form, size):
    p = Product(form, size, sum(size))
    for g, got, a, b in p.parts(p.run(lib)):
        assert (got == rounded(a @ b.T)).all(), g


@pytest.mark.parametrize("bn", PAIRS["dense"])
def test_c_may_be_d(lib, bn):
    for _ in range(3):
        check_exact(lib, *pair(1, *PAIRS["dense"][bn]), True, alias=True)


@pytest.mark.parametrize("form, size", SPECIAL)
def test_wide_scales(lib, form, size):
    p = Product(form, size, 2, (100, 140), (110, 150))
    for _, got, a, b in p.parts(p.run(lib)):
        want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
        assert (np.abs(floats(got) - want) <= 2.0 ** -8 * np.abs(want) + (p.K // 64) * 2.0 ** -22 * mag).all()


@pytest.mark.parametrize("form, size", SPECIAL)
def test_a_scale_that_is_not_a_number(lib, form, size):
    p = Product(form, size, 3)
    g = max(range(len(p.rows)), key=lambda i: len(p.rows[i]))
    row, column = p.rows[g][len(p.rows[g]) // 2], 17
    places = (p.operand(g).exps, row, 3), (p.b[g].exps, column, p.K // 32 - 1)
    for e, r, k in places:
        e[r, k] = 255
    p.repack()
    bits = p.run(lib)
    for e, r, k in places:
        e[r, k] = 127
    p.repack()
    for i, got, a, b in p.parts(bits):
        bad = np.zeros(got.shape, bool)
        if i == g:
            bad[p.rows[g] == row], bad[:, column] = True, True
        want = a @ b.T
        assert np.isnan(floats(got)[bad]).all() and (got[~bad] == bits_of(want[~bad])).all()


@pytest.mark.parametrize("form, size", SPECIAL)
def test_scales_at_the_ends(lib, form, size):
    # 2^-127 * 2^127, and results that FP32 rounds to infinity or to 0
    p = Product(form, size, 4)
    for o in p.a:
        o.packed[:], o.exps[0::2], o.exps[1::2] = 0x22, 0, 254          # all ones
    for o in p.b:
        o.packed[:], o.exps[:p.N // 2], o.exps[p.N // 2:] = 0x22, 254, 0
    p.repack()
    for g, got, _, _ in p.parts(p.run(lib)):
        low, left = p.rows[g] % 2 == 0, np.arange(p.N) < p.N // 2
        want = np.where(low[:, None] == left, float(p.K), np.where(left, np.inf, 0.0))
        assert (floats(got) == want).all()


@pytest.mark.parametrize("form, size", SPECIAL)
def test_every_place_of_k(lib, form, size):
    # one nonzero in each row of A picks a column of B
    p = Product(form, size, 5, (122, 131), (120, 134))
    for o in p.a:
        codes = np.zeros((p.M, p.K), np.uint8)
        codes[np.arange(p.M), np.arange(p.M) * 7 % p.K] = 2              # 1.0
        o.packed = W.pack_fp4(codes)
    for g, got, a, b in p.parts(p.run(lib)):
        assert (got == rounded(a @ b.T)).all(), g


@pytest.mark.parametrize("bn", PAIRS["dense"])
def test_addends_that_are_not_finite(lib, bn):
    M, N, K = PAIRS["dense"][bn]
    a, b = pair(6, M, N, K)
    c = torch.zeros(M, N, device="cuda", dtype=BF16)
    c[1, 3], c[2, 5], c[M - 1, N - 1] = float("nan"), float("inf"), -float("inf")
    d = sentinel_like((M, N))
    lib.dg_fp4_gemm_nt(dev(a.packed), dev(a.sf), dev(b.packed), dev(b.sf), c, d)
    d = d.float().cpu()
    assert d[1, 3].isnan() and d[2, 5] == float("inf") and d[M - 1, N - 1] == -float("inf") and int((~d.isfinite()).sum()) == 3


# kernels that test_fp4_gemm_gpu.py's captures and waits do not reach
OTHERS = [("dense", PAIRS["dense"][128]), ("dense", (100, 4096, 8192)), ("dense", (402, 2112, 14080)), ("contiguous", PAIRS["contiguous"][256]),
          ("contiguous", PAIRS["contiguous"][384]), ("masked", PAIRS["masked"][256]), ("masked", PAIRS["masked"][384])]


@pytest.mark.parametrize("form, size", OTHERS)
def test_captured_replayed_and_a_wait_that_runs_out(lib, form, size):
    call, d = Product(form, size, 7).call(lib)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    want = bf16_bits(d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(s)
    untouched = sentinel_like(d.shape)
    for _ in range(2):
        d.copy_(untouched)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert (bf16_bits(d) == want).all()
    lib.dg_set_debug(1, 20_000_000)
    try:
        call(s)
        assert lib.dg_get_device_status(s) == 5
    finally:
        lib.dg_set_debug(0)
    d.copy_(untouched)
    torch.cuda.synchronize()
    call(s)
    assert lib.dg_get_device_status(s) == 0
    assert (bf16_bits(d) == want).all()
