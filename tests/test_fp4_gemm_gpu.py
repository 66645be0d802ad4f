"""The products of two FP4 operands against the FP64 oracle.

Exact cases: codes are random, scales within a factor of 2^d, so that every term is a whole multiple of one unit and the
sum of all their magnitudes stays below 2^24 of it: FP32 holds every partial sum in any order, and D has to be the one
rounding of the exact sum to BF16, bit for bit. Other cases: scales over a wide range; each of the K / 64 instructions
rounds a partial sum, by 2^-22 of the terms' magnitudes at most, and D is rounded to 2^-8."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.four_bit as F
import workloads as W
from gpu_util import bf16_bits, dev, sentinel_like

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    L.dg_get_device_status()
    return L


class Operand:
    """Random codes [rows, K] and scale exponents in [lo, hi]."""

    def __init__(self, rng, rows, K, lo, hi):
        self.packed = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
        self.exps = rng.integers(lo, hi + 1, (rows, K // 32)).astype(np.uint8)
        self.sf = W.pack_sf(self.exps)


def spread(K):
    """d with 36 * 4 (in units of 1/4) * 2^d * K < 2^24, split over both operands."""
    return max(0, int(np.floor(np.log2(2.0 ** 24 / (144 * K)))))


def bits_of(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(BF16).view(torch.int16).numpy().view(np.uint16)


def rounded(exact):
    """BF16 bits of values that FP32 holds."""
    assert (exact == exact.astype(np.float32)).all()
    return bits_of(exact)


def pair(seed, M, N, K, exact=True):
    rng = np.random.default_rng(seed)
    if not exact:
        return Operand(rng, M, K, 100, 140), Operand(rng, N, K, 110, 150)
    d = spread(K)
    a, b = Operand(rng, M, K, 127, 127 + d // 2), Operand(rng, N, K, 127, 127 + d - d // 2)
    return a, b


def run_dense(L, a, b, c=None, alias=False):
    d = c if alias else sentinel_like((len(a.packed), len(b.packed)))
    assert L.dg_fp4_gemm_nt(dev(a.packed), dev(a.sf), dev(b.packed), dev(b.sf), c, d) is d
    torch.cuda.synchronize()
    return d


def check_exact(L, a, b, with_c, seed=0, alias=False):
    want = F.gemm(a.packed, a.sf, b.packed, b.sf)
    c = None
    if with_c:
        # whole numbers of eight bits, which the sums' unit divides
        c64 = np.random.default_rng(seed).integers(-255, 256, want.shape).astype(np.float64)
        c, want = torch.from_numpy(c64).cuda().to(BF16), want + c64
    d = run_dense(L, a, b, c, alias)
    assert (bf16_bits(d) == rounded(want)).all()
    assert L.dg_get_device_status() == 0


# sizes that take each way of the dispatch: tiles of 64 to 192 columns with K whole or shared out, CTA pairs with 128 and 256
SIZES = [(1, 16, 128), (1, 16, 896), (3, 48, 256), (5, 400, 512), (130, 64, 640), (300, 2048, 384), (32, 2352, 1024), (7, 2048, 4096), (1, 5152, 1408),
         (128, 5504, 1536), (16, 5504, 2048), (100, 9984, 256), (9, 14000, 128), (128, 24576, 512), (700, 7168, 512), (140, 19872, 128), (515, 4096, 1152),
         (1000, 4096, 640), (1030, 2576, 2048), (2050, 2064, 384), (4096, 2048, 1024)]


@pytest.mark.parametrize("M, N, K", SIZES)
@pytest.mark.parametrize("with_c", [False, True])
def test_dense_exact(lib, M, N, K, with_c):
    a, b = pair(M + N + K, M, N, K)
    check_exact(lib, a, b, with_c, seed=M)


@pytest.mark.parametrize("M, N, K", [(33, 400, 1024), (600, 4096, 512)])
def test_c_may_be_d(lib, M, N, K):
    a, b = pair(1, M, N, K)
    check_exact(lib, a, b, True, alias=True)


def test_random_sizes_exact(lib):
    rng = np.random.default_rng(77)
    for i in range(40):
        M, N, K = int(np.exp(rng.uniform(0, 7))), 16 * int(np.exp(rng.uniform(0, 5.3))), 128 * int(np.exp(rng.uniform(0, 3.2)))
        a, b = pair(100 + i, M, N, K)
        check_exact(lib, a, b, bool(i % 2), seed=i)


@pytest.mark.parametrize("M, N, K", [(1, 64, 256), (50, 512, 4096), (300, 4096, 2048), (1100, 2048, 1024)])
def test_wide_scales(lib, M, N, K):
    a, b = pair(2, M, N, K, exact=False)
    want, mag = F.gemm(a.packed, a.sf, b.packed, b.sf), F.gemm_magnitude(a.packed, a.sf, b.packed, b.sf)
    got = run_dense(lib, a, b).double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (K // 64) * 2.0 ** -22 * mag).all()


def test_every_code_and_scale_place(lib):
    # one nonzero in A picks a column of B: each place of K, each code, each scale byte comes back by itself
    M, N, K = 256, 32, 256
    rng = np.random.default_rng(3)
    b = Operand(rng, N, K, 120, 134)
    a = Operand(rng, M, K, 127, 127)
    codes = np.zeros((M, K), np.uint8)
    codes[np.arange(M), np.arange(M)] = 2                            # 1.0
    a.packed, a.exps = W.pack_fp4(codes), rng.integers(122, 132, (M, K // 32)).astype(np.uint8)
    a.sf = W.pack_sf(a.exps)
    check_exact(lib, a, b, False)


def test_scales_at_the_ends(lib):
    # 2^-127 * 2^127, and results that FP32 rounds to infinity or to 0
    M, N, K = 4, 16, 128
    a, b = pair(4, M, N, K)
    a.packed[:] = 0x22                                              # all ones
    b.packed[:] = 0x22
    a.exps[:] = np.array([0, 254, 0, 254], np.uint8)[:, None]
    b.exps[:8], b.exps[8:] = 254, 0
    a.sf, b.sf = W.pack_sf(a.exps), W.pack_sf(b.exps)
    got = run_dense(lib, a, b).double().cpu().numpy()
    want = np.zeros((4, 16))
    want[0::2, :8], want[1::2, 8:], want[1::2, :8], want[0::2, 8:] = 128, 128, np.inf, 0
    assert (got == want).all()


def test_a_scale_that_is_not_a_number(lib):
    for M, N, K in ((6, 64, 512), (400, 4096, 512)):
        a, b = pair(5, M, N, K)
        a.exps[M // 2, 3], b.exps[17, K // 32 - 1] = 255, 255
        a.sf, b.sf = W.pack_sf(a.exps), W.pack_sf(b.exps)
        got = run_dense(lib, a, b).double().cpu().numpy()
        bad = np.zeros((M, N), bool)
        bad[M // 2], bad[:, 17] = True, True
        a.exps[M // 2, 3], b.exps[17, K // 32 - 1] = 127, 127
        want = F.gemm(a.packed, W.pack_sf(a.exps), b.packed, W.pack_sf(b.exps))
        assert np.isnan(got[bad]).all() and (bits_of(got[~bad]) == rounded(want[~bad])).all()


def test_addends_that_are_not_finite(lib):
    for M, N, K in ((6, 64, 512), (400, 4096, 512)):
        a, b = pair(6, M, N, K)
        c = torch.zeros(M, N, device="cuda", dtype=BF16)
        c[1, 3], c[2, 5], c[M - 1, N - 1] = float("nan"), float("inf"), -float("inf")
        d = run_dense(lib, a, b, c).float().cpu()
        assert d[1, 3].isnan() and d[2, 5] == float("inf") and d[M - 1, N - 1] == -float("inf") and int((~d.isfinite()).sum()) == 3


# --------------------------------------------------------------------------------------
# grouped forms
# --------------------------------------------------------------------------------------

def stacked(ops):
    return dev(np.stack([o.packed for o in ops])), dev(np.stack([o.sf for o in ops]))


def check_masked(L, G, max_m, N, K, counts, seed=0, status=0):
    rng = np.random.default_rng(seed)
    s = spread(K)
    a, b = [Operand(rng, max_m, K, 127, 127 + s // 2) for _ in range(G)], [Operand(rng, N, K, 127, 127 + s - s // 2) for _ in range(G)]
    da, dsa = stacked(a)
    db, dsb = stacked(b)
    d = sentinel_like((G, max_m, N))
    before = bf16_bits(d).copy()
    assert L.dg_m_grouped_fp4_gemm_nt_masked(da, dsa, db, dsb, d, dev(np.array(counts, np.int32))) is d
    assert L.dg_get_device_status() == status
    got = bf16_bits(d)
    for g, c in enumerate(counts):
        c = min(max(c, 0), max_m)
        want = rounded(F.gemm(a[g].packed, a[g].sf, b[g].packed, b[g].sf)[:c])
        assert (got[g, :c] == want).all() and (got[g, c:] == before[g, c:]).all(), g


@pytest.mark.parametrize("G, max_m, N, K, counts", [
    (1, 1, 16, 128, [1]), (3, 7, 64, 256, [0, 7, 3]), (4, 128, 272, 384, [128, 0, 1, 127]), (4, 256, 528, 640, [256, 129, 128, 200]),
    (5, 300, 144, 512, [300, 0, 257, 256, 31]), (2, 517, 2048, 256, [517, 260]), (6, 40, 7168, 128, [40, 0, 0, 13, 1, 40]), (3, 130, 512, 2048, [0, 0, 0]),
    (32, 20, 256, 256, [20, 3] * 16)])
def test_masked(lib, G, max_m, N, K, counts):
    check_masked(lib, G, max_m, N, K, counts, seed=G + max_m)


def test_masked_counts_out_of_range(lib):
    check_masked(lib, 3, 40, 128, 256, [41, -5, 7], status=6)


def test_masked_many_groups(lib):
    # more groups than the counts that a CTA keeps
    rng = np.random.default_rng(8)
    check_masked(lib, 1100, 3, 16, 128, rng.integers(0, 4, 1100).tolist())


def test_masked_rows_past_32_bits(lib):
    # D's last group begins past 2^31 elements
    rng = np.random.default_rng(12)
    G, max_m, N, K = 4, 45001, 16384, 128
    a, b = torch.zeros(G, max_m, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(G, N, K // 2, dtype=torch.uint8, device="cuda")
    sfa, sfb = (torch.full((G, 1, up), 0x7F7F7F7F, dtype=torch.int32, device="cuda") for up in (45004, N))
    rows, columns = rng.integers(0, 256, (300, K // 2), dtype=np.uint8), rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    a[3, :300], b[3] = dev(rows), dev(columns)
    d = torch.full((G, max_m, N), 7.0, dtype=BF16, device="cuda")
    lib.dg_m_grouped_fp4_gemm_nt_masked(a, sfa, b, sfb, d, dev(np.array([0, 1, 0, 300], np.int32)))
    assert lib.dg_get_device_status() == 0
    ones = W.pack_sf(np.full((N, 4), 127, np.uint8))
    want = F.gemm(rows, ones[:, :300], columns, ones)
    assert (bf16_bits(d[3, :300]) == rounded(want)).all()
    assert (d[3, 300:400] == 7).all() and (d[1, 0] == 0).all() and (d[1, 1:100] == 7).all() and (d[2, :100] == 7).all()


def check_contiguous(L, sizes, N, K, G=None, seed=0, hole=None, align=128):
    rng = np.random.default_rng(seed)
    G = len(sizes) if G is None else G
    s = spread(K)
    index = []
    for e, rows in enumerate(sizes):
        index += [e] * rows + [-1] * (-rows % align)
    if hole is not None:
        index += [-1] * hole                             # blocks of nothing but padding
    index = np.array(index, np.int32)
    a, b = Operand(rng, len(index), K, 127, 127 + s // 2), [Operand(rng, N, K, 127, 127 + s - s // 2) for _ in range(G)]
    db, dsb = stacked(b)
    d = sentinel_like((len(index), N))
    before = bf16_bits(d).copy()
    assert L.dg_m_grouped_fp4_gemm_nt_contiguous(dev(a.packed), dev(a.sf), db, dsb, d, dev(index)) is d
    assert L.dg_get_device_status() == 0
    got = bf16_bits(d)
    av = F.values(a.packed, a.sf)
    for e in range(len(sizes)):
        at = index == e
        assert (got[at] == rounded(av[at] @ F.values(b[e].packed, b[e].sf).T)).all(), e
    assert (got[index < 0] == before[index < 0]).all()


@pytest.mark.parametrize("sizes, N, K", [([1], 16, 128), ([128], 64, 256), ([129, 5], 272, 384), ([0, 300, 0, 128, 1], 528, 640), ([256, 512, 130, 700], 144, 512),
                                         ([60] * 16, 2048, 256), ([1000, 24], 4096, 1152)])
def test_contiguous(lib, sizes, N, K):
    check_contiguous(lib, sizes, N, K, seed=len(sizes))


def test_contiguous_padding_blocks_and_experts_without_rows(lib):
    check_contiguous(lib, [200, 0, 50], 256, 256, G=9, hole=384)
    check_contiguous(lib, [200, 30], 256, 256, align=256)


def test_contiguous_long_runs(lib):
    # runs that pass the 32 blocks that are looked at together, of odd and even lengths
    check_contiguous(lib, [128 * 33, 5, 128 * 40 + 3, 128 * 31, 128 * 2], 144, 128)


def test_contiguous_blocks_of_every_neighbour(lib):
    # every order of experts and padding over two neighbouring blocks, in steps of 256 rows and across them
    rng = np.random.default_rng(20)
    N, K, G = 400, 256, 3
    blocks = rng.permutation([e for e in (-1, 0, 1, 2) for _ in range(9)])
    s = spread(K)
    a, b = Operand(rng, 128 * len(blocks), K, 127, 127 + s // 2), [Operand(rng, N, K, 127, 127 + s - s // 2) for _ in range(G)]
    index = np.repeat(blocks, 128).astype(np.int32)
    index[128 * 5 + 100:128 * 6] = -1                    # padding rows at a block's end
    db, dsb = stacked(b)
    d = sentinel_like((len(index), N))
    before = bf16_bits(d).copy()
    lib.dg_m_grouped_fp4_gemm_nt_contiguous(dev(a.packed), dev(a.sf), db, dsb, d, dev(index))
    assert lib.dg_get_device_status() == 0
    got, av = bf16_bits(d), F.values(a.packed, a.sf)
    for e in range(G):
        at = index == e
        assert (got[at] == rounded(av[at] @ F.values(b[e].packed, b[e].sf).T)).all()
    assert (got[index < 0] == before[index < 0]).all()


def test_contiguous_all_padding(lib):
    d = sentinel_like((256, 64))
    before = d.clone()
    a, b = pair(9, 256, 64, 128)
    lib.dg_m_grouped_fp4_gemm_nt_contiguous(dev(a.packed), dev(a.sf), dev(b.packed[None]), dev(b.sf[None]), d, torch.full((256,), -1, dtype=torch.int32, device="cuda"))
    assert lib.dg_get_device_status() == 0 and torch.equal(d.view(torch.int16), before.view(torch.int16))


def test_contiguous_rows_of_no_expert(lib):
    # M_total that is no multiple of 128 or of 4, and indices that break the layout
    a, b = pair(10, 131, 64, 128)
    index = np.zeros(131, np.int32)
    d = sentinel_like((131, 64))
    lib.dg_m_grouped_fp4_gemm_nt_contiguous(dev(a.packed), dev(a.sf), dev(b.packed[None]), dev(b.sf[None]), d, dev(index))
    assert lib.dg_get_device_status() == 0
    want = rounded(F.gemm(a.packed, a.sf, b.packed, b.sf))
    assert (bf16_bits(d) == want).all()
    index[5], index[128] = 3, 7                          # another expert inside a block; an expert that does not exist
    d = sentinel_like((131, 64))
    before = bf16_bits(d).copy()
    lib.dg_m_grouped_fp4_gemm_nt_contiguous(dev(a.packed), dev(a.sf), dev(b.packed[None]), dev(b.sf[None]), d, dev(index))
    assert lib.dg_get_device_status() == 6
    ok = np.ones(131, bool)
    ok[5], ok[128:] = False, False
    got = bf16_bits(d)
    assert (got[ok] == want[ok]).all() and (got[~ok] == before[~ok]).all()


# --------------------------------------------------------------------------------------
# streams, graphs, settings, waits that run out
# --------------------------------------------------------------------------------------

def forms(L):
    """(name, call(stream), output) of each form and way."""
    out = []
    for M, N, K in ((5, 400, 512), (32, 2352, 1024), (7, 2048, 4096), (16, 5504, 2048), (700, 7168, 512), (1000, 4096, 640)):
        a, b = pair(M, M, N, K)
        ops = dev(a.packed), dev(a.sf), dev(b.packed), dev(b.sf)
        c, d = torch.ones(M, N, device="cuda", dtype=BF16), torch.empty(M, N, device="cuda", dtype=BF16)
        out.append((f"dense {M} {N} {K}", lambda s, ops=ops, c=c, d=d: L.dg_fp4_gemm_nt(*ops, c, d, stream=s), d))
    a, b = pair(11, 3 * 256, 512, 256)
    ops = dev(a.packed.reshape(3, 256, -1)), dev(np.stack([W.pack_sf(a.exps[256 * g:256 * g + 256]) for g in range(3)]))
    wide = dev(np.stack([b.packed] * 3)), dev(np.stack([b.sf] * 3))
    d1, d2 = (torch.zeros(768, 512, device="cuda", dtype=BF16) for _ in range(2))
    counts, index = dev(np.array([256, 0, 130], np.int32)), dev(np.repeat(np.array([0, 1, 2], np.int32), 256))
    flat = dev(a.packed), dev(a.sf)
    out.append(("masked", lambda s: L.dg_m_grouped_fp4_gemm_nt_masked(*ops, *wide, d1.view(3, 256, 512), counts, stream=s), d1))
    out.append(("contiguous", lambda s: L.dg_m_grouped_fp4_gemm_nt_contiguous(*flat, *wide, d2, index, stream=s), d2))
    return out


def test_captured_and_replayed(lib):
    for name, call, d in forms(lib):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        call(s)
        s.synchronize()
        want = d.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(s)
        for _ in range(2):
            d.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(d.view(torch.int16), want.view(torch.int16)), name
    assert lib.dg_get_device_status() == 0


def test_the_same_with_and_without_early_launch_and_on_few_sms(lib):
    s = torch.cuda.current_stream()
    for name, call, d in forms(lib):
        call(s)
        want = d.clone()
        for set_up, undo in ((lambda: lib.dg_set_pdl(False), lambda: lib.dg_set_pdl(True)), (lambda: lib.dg_set_num_sms(20), lambda: lib.dg_set_num_sms(0)),
                             (lambda: lib.dg_set_num_sms(1), lambda: lib.dg_set_num_sms(0))):
            set_up()
            try:
                d.zero_()
                call(s)
                torch.cuda.synchronize()
                assert torch.equal(d.view(torch.int16), want.view(torch.int16)), name
            finally:
                undo()
    assert lib.dg_get_device_status() == 0


def test_two_streams_at_once(lib):
    jobs = [(call, d, torch.cuda.Stream()) for _, call, d in forms(lib)]
    torch.cuda.synchronize()
    for call, d, s in jobs:
        call(s)
    torch.cuda.synchronize()
    want = [d.clone() for _, d, _ in jobs]
    for _, d, _ in jobs:
        d.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for call, d, s in jobs:
            call(s)
    torch.cuda.synchronize()
    assert all(torch.equal(d.view(torch.int16), w.view(torch.int16)) for (_, d, _), w in zip(jobs, want))
    assert lib.dg_get_device_status() == 0


def test_a_wait_that_runs_out(lib):
    s = torch.cuda.current_stream()
    for name, call, d in forms(lib):
        call(s)
        want = d.clone()
        lib.dg_set_debug(1, 20_000_000)
        try:
            call(s)
            assert lib.dg_get_device_status() == 5, name
        finally:
            lib.dg_set_debug(0)
        call(s)
        assert lib.dg_get_device_status() == 0
        assert torch.equal(d.view(torch.int16), want.view(torch.int16)), name
