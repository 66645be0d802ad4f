"""The mixture-of-experts layer for a few tokens against the FP64 oracle.

Tolerances, from the arithmetic: products of E4M3 and E2M1 values are exact in FP32; a dot
product accumulates in FP32 in chains of at most H / 128 + 8 roundings or truncations at 2^-23, so it is
within 2^-15 of the sum of its terms' magnitudes. The inner values are held to 11 bits or more under a
shared scale: 2^-11 of themselves. The oracle carries both through to y; storing y in BF16 adds 2^-8 of it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.layers as OL
import workloads as W

pytestmark = pytest.mark.gpu

BF16_REL = 2.0 ** -8


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    return L


def _packed(exps, fmt):
    """Exponents [N, groups] of one expert -> its packed words."""
    if fmt == "e4m3":
        return W.pack_sf(exps)
    N, kb = exps.shape
    out = np.zeros((kb // 4, 4 * (-(-N // 4)), 4), np.uint8)
    out[:, :N] = exps.reshape(N, kb // 4, 4).transpose(1, 0, 2)
    return out.reshape(kb // 4, -1).view(np.int32)


class Layer:
    def __init__(self, T, E, k, H, I, fmt, seed, c=True):
        rng = np.random.default_rng(seed)
        self.fmt, self.T, self.E, self.k, self.H, self.I = fmt, T, E, k, H, I
        self.x, ex = W.quantize_rows(rng.normal(size=(T, H)).astype(np.float32) * np.exp2(rng.integers(-3, 4, (T, 1))).astype(np.float32))
        self.sfx = W.pack_sf(ex)
        self.w13, self.sf13 = self._weights(rng, E, 2 * I, H)
        self.w2, self.sf2 = self._weights(rng, E, H, I)
        self.ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        self.weights = rng.random((T, k)).astype(np.float32)
        self.c = W.to_bf16_bits(rng.normal(size=(T, H)).astype(np.float32)) if c else None

    def _weights(self, rng, E, N, K):
        lo = 114 if self.fmt == "e4m3" else 118
        if self.fmt == "e4m3":
            w = rng.integers(0, 256, (E, N, K), dtype=np.uint8)
            w[(w & 0x7F) == 0x7F] = 0                        # no NaN codes
            w[(w & 0x7F) > 0x70] &= 0xBF                     # few large ones
            e = rng.integers(lo - 4, lo, (E, -(-N // 128), K // 128)).astype(np.uint8)
        else:
            w = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
            e = rng.integers(lo, lo + 6, (E, N, K // 32)).astype(np.uint8)
        return w, np.stack([_packed(m, self.fmt) for m in e])

    def run(self, L, y=None, stream=None, **over):
        d = {n: torch.from_numpy(np.ascontiguousarray(over.get(n, getattr(self, n)))).cuda()
             for n in ("x", "sfx", "w13", "sf13", "w2", "sf2", "ids", "weights")}
        c = None if self.c is None else torch.from_numpy(self.c.view(np.int16)).view(torch.bfloat16).cuda()
        if y is None:
            y = torch.full((self.T, self.H), float("nan"), dtype=torch.bfloat16, device="cuda")
        fn = L.dg_moe_fp8_few_tokens if self.fmt == "e4m3" else L.dg_moe_fp8_fp4_few_tokens
        fn(*d.values(), c, y, stream=stream)
        torch.cuda.synchronize()
        return y

    def oracle(self, **over):
        a = {n: over.get(n, getattr(self, n)) for n in ("x", "sfx", "w13", "sf13", "w2", "sf2", "ids", "weights")}
        c = None if self.c is None else (self.c.astype(np.uint32) << 16).view(np.float32)
        bound = {"dot": 2.0 ** -15, "inner": 2.0 ** -11}
        return OL.moe_layer(*a.values(), c, self.fmt, bound), bound["y"]


def check(y, want, err):
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= 1.01 * (BF16_REL * np.abs(want) + err)).all(), np.abs(got - want).max()
    # and in the mean: BF16's rounding is at most 2^-8 / sqrt(3) of the values, the inner values' far below
    assert np.linalg.norm(got - want) <= 0.75 * BF16_REL * np.linalg.norm(want)


SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (2, 4, 4, 640, 384), (8, 8, 2, 384, 256), (9, 3, 3, 512, 128), (17, 5, 4, 1920, 128),
          (32, 2, 2, 256, 256), (32, 40, 8, 128, 640), (31, 1, 1, 768, 128), (5, 300, 16, 128, 128), (3, 6, 2, 4224, 256), (16, 7, 1, 256, 2176)]


@pytest.mark.parametrize("T, E, k, H, I", SHAPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_layer(lib, T, E, k, H, I, fmt):
    p = Layer(T, E, k, H, I, fmt, seed=T * 31 + E, c=(T + H) % 2 == 0)
    check(p.run(lib), *p.oracle())
    assert lib.dg_get_device_status() == 0


@pytest.mark.parametrize("T, E, k, H, I", [(32, 40, 8, 128, 640), (32, 64, 8, 256, 384), (8, 64, 8, 128, 640), (20, 50, 6, 384, 896), (7, 100, 9, 512, 640)])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_short_rows_many_units(lib, T, E, k, H, I, fmt):
    # a row is one to four pieces and a block has several units: the copies run past unit boundaries.
    # No addend, so that the experts' part alone is judged.
    p = Layer(T, E, k, H, I, fmt, seed=T + H + I, c=False)
    check(p.run(lib), *p.oracle())


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_empty_slots_duplicates_and_bad_ids(lib, fmt):
    p = Layer(12, 5, 4, 256, 128, fmt, seed=7)
    p.ids[0] = -1                                            # a token without an expert
    p.ids[1] = [3, 3, -1, 3]                                 # one expert three times
    p.ids[2, 1] = -1
    p.weights[3] = 0                                         # weights of 0, of either sign, large
    p.weights[4] = [-1.0, 1e4, 0.0, -2.0]
    check(p.run(lib), *p.oracle())
    assert lib.dg_get_device_status() == 0
    bad = p.ids.copy()
    bad[5, 0], bad[6, 2] = 5, -7
    y = p.run(lib, ids=bad)
    assert lib.dg_get_device_status() == 6 and lib.dg_get_device_status() == 0
    check(y, *p.oracle(ids=np.where((bad < 0) | (bad >= 5), -1, bad)))
    none = np.full_like(p.ids, -1)
    y = p.run(lib, ids=none)
    assert (y.cpu().view(torch.int16).numpy() == p.c.view(np.int16)).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_other_experts_and_tokens_do_not_reach_a_token(lib, fmt):
    p = Layer(10, 4, 2, 256, 256, fmt, seed=8)
    p.ids[:] = [[0, 1]] * 5 + [[2, 3]] * 5
    p.ids[7] = [1, 2]
    base = p.run(lib)
    touched = (p.ids == 3).any(1)
    # expert 3 becomes NaN: through its scales (code 255) in both matrices
    sf13, sf2 = p.sf13.copy(), p.sf2.copy()
    sf13[3], sf2[3] = -1, -1
    y = p.run(lib, sf13=sf13, sf2=sf2)
    assert y[torch.from_numpy(touched)].isnan().all() and torch.equal(y[torch.from_numpy(~touched)], base[torch.from_numpy(~touched)])
    # token 2 becomes NaN
    x = p.x.copy()
    x[2] = 0x7F
    y = p.run(lib, x=x)
    others = torch.arange(10) != 2
    assert y[2].isnan().all() and torch.equal(y[others], base[others])


def test_inner_values_far_apart(lib):
    # the experts' inner values span 2^40 between blocks of 64 columns: each block has its own scale
    p = Layer(4, 2, 1, 256, 256, "e4m3", seed=9, c=False)
    e = np.full((2, 4, 2), 116, np.uint8)
    e[:, 1], e[:, 3] = 136, 136                              # the second 128 columns: gate and up 2^20 times the first's
    p.sf13 = np.stack([W.pack_sf(m) for m in e])
    e2 = np.full((2, 2, 2), 114, np.uint8)
    e2[:, :, 1] = 74                                         # and W2 brings them back
    p.sf2 = np.stack([W.pack_sf(m) for m in e2])
    check(p.run(lib), *p.oracle())


def test_scale_codes_at_the_ends(lib):
    # code 0 is 2^-127 and stays a value; products that underflow are 0
    p = Layer(2, 2, 1, 128, 128, "e4m3", seed=10)
    sf = p.sf13.copy()
    sf[:] = 0
    y = p.run(lib, sf13=sf)
    assert (y.cpu().view(torch.int16).numpy() == p.c.view(np.int16)).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_same_bits_streams_graph_in_place_and_pdl(lib, fmt):
    p = Layer(11, 6, 3, 512, 384, fmt, seed=11)
    base = p.run(lib)
    fn = lib.dg_moe_fp8_few_tokens if fmt == "e4m3" else lib.dg_moe_fp8_fp4_few_tokens
    ops = [torch.from_numpy(getattr(p, n)).cuda() for n in ("x", "sfx", "w13", "sf13", "w2", "sf2", "ids", "weights")]
    c = torch.from_numpy(p.c.view(np.int16)).view(torch.bfloat16).cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    try:
        for pdl in (0, 1):
            lib.dg_set_pdl(pdl)
            y = c.clone()
            torch.cuda.synchronize()
            for _ in range(3):                               # back to back on one workspace
                fn(*ops, c, y, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(y, base)
    finally:
        lib.dg_set_pdl(1)
    y = c.clone()
    torch.cuda.synchronize()
    fn(*ops, y, y, stream=s)                                 # in place
    torch.cuda.synchronize()
    assert torch.equal(y, base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fn(*ops, c, y, stream=s)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, base)
    lib.dg_set_num_sms(5)
    try:
        check(p.run(lib), *p.oracle())
    finally:
        lib.dg_set_num_sms(0)


def test_a_stale_workspace_and_a_gemm_between(lib):
    # calls of other sizes and a stream-K GEMM share the stream's workspace
    small, large = Layer(3, 4, 2, 256, 128, "e4m3", seed=12), Layer(32, 8, 4, 384, 512, "e2m1", seed=13)
    first = small.run(lib), large.run(lib)
    g = W.make_dense(128, 512, 4096, seed=1)
    d = torch.empty(128, 512, dtype=torch.bfloat16, device="cuda")
    ops = [torch.from_numpy(v).cuda() for v in (g.a, g.sfa, g.b, g.sfb)]
    lib.dg_fp8_gemm_nt(*ops, None, d)
    before = d.clone()
    assert torch.equal(large.run(lib), first[1]) and torch.equal(small.run(lib), first[0])
    lib.dg_fp8_gemm_nt(*ops, None, d)
    assert torch.equal(d, before) and lib.dg_get_device_status() == 0


def test_experts_past_four_gib(lib):
    # the last of many experts lies past 2^32 bytes: the same bits as alone
    T, H, I, E = 2, 7168, 2048, 180
    g = torch.Generator(device="cuda").manual_seed(1)
    u8 = lambda *s: torch.randint(0, 0x70, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    w13, w2 = torch.zeros(E, 2 * I, H, dtype=torch.uint8, device="cuda"), torch.zeros(E, H, I, dtype=torch.uint8, device="cuda")
    w13[-1], w2[-1] = u8(2 * I, H), u8(H, I)
    sf13 = torch.full((E,) + lib.sf_shape(2 * I // 128, H), 0x70707070, dtype=torch.int32, device="cuda")
    sf2 = torch.full((E,) + lib.sf_shape(H // 128, I), 0x70707070, dtype=torch.int32, device="cuda")
    x, sfx = u8(T, H), torch.full(lib.sf_shape(T, H), 0x70707070, dtype=torch.int32, device="cuda")
    w = torch.rand(T, 1, device="cuda", generator=g)
    out = []
    for e0, e in ((0, E - 1), (E - 1, 0)):
        ids = torch.full((T, 1), e, dtype=torch.int32, device="cuda")
        y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        lib.dg_moe_fp8_few_tokens(x, sfx, w13[e0:], sf13[e0:], w2[e0:], sf2[e0:], ids, w, None, y)
        out.append(y)
    assert torch.equal(*out) and out[0].abs().sum() > 0


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_a_wait_that_runs_out_is_reported(lib, fmt):
    p = Layer(6, 4, 2, 512, 384, fmt, seed=17)
    base = p.run(lib)
    lib.dg_set_debug(1, 20_000_000)          # no weights are copied; waits give up after 20 ms
    try:
        p.run(lib)
        assert lib.dg_get_device_status() == 5   # DG_ERR_TIMEOUT
    finally:
        lib.dg_set_debug(0, 0)
    assert torch.equal(p.run(lib), base) and lib.dg_get_device_status() == 0


@pytest.mark.parametrize("T, E, k", [(32, 1, 1), (32, 2, 2), (11, 1, 1), (16, 3, 2), (25, 2, 1), (32, 3, 1)])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_many_tokens_of_an_expert(lib, T, E, k, fmt):
    # more of them than one MMA takes as columns, in either product
    p = Layer(T, E, k, 384, 256, fmt, seed=T + E, c=False)
    check(p.run(lib), *p.oracle())


def test_binding_refuses(lib):
    p = Layer(2, 3, 2, 128, 128, "e4m3", seed=14)
    d = {n: torch.from_numpy(getattr(p, n)).cuda() for n in ("x", "sfx", "w13", "sf13", "w2", "sf2", "ids", "weights")}
    y = torch.empty(2, 128, dtype=torch.bfloat16, device="cuda")

    def call(y=y, c=None, fn=lib.dg_moe_fp8_few_tokens, **over):
        fn(*{**d, **over}.values(), c, y)

    call()
    for bad in (dict(x=d["x"].float()), dict(ids=d["ids"].long()), dict(weights=d["weights"][:1]), dict(w13=d["w13"][:, :200].contiguous()),
                dict(sf2=d["sf2"][:2].contiguous()), dict(sfx=d["sfx"][:, :2].contiguous()), dict(w2=d["w2"].cpu()),
                dict(y=y.float()), dict(c=y[:1]), dict(fn=lib.dg_moe_fp8_fp4_few_tokens)):
        with pytest.raises(ValueError):
            call(**bad)
    f = Layer(2, 3, 2, 128, 128, "e2m1", seed=14)
    d4 = {n: torch.from_numpy(getattr(f, n)).cuda() for n in ("w13", "sf13", "w2", "sf2")}
    call(fn=lib.dg_moe_fp8_fp4_few_tokens, **d4)
    off16 = torch.empty(3 * 128 * 64 + 16, dtype=torch.uint8, device="cuda")[16:].view(3, 128, 64)
    with pytest.raises(lib.DGError, match="MISALIGNED"):
        call(fn=lib.dg_moe_fp8_fp4_few_tokens, **{**d4, "w2": off16})
    odd = torch.empty(3 * 256 * 128 + 8, dtype=torch.uint8, device="cuda")[8:].view(3, 256, 128)
    with pytest.raises(lib.DGError, match="MISALIGNED"):
        call(w13=odd)
    q = Layer(33, 3, 2, 128, 128, "e4m3", seed=15)
    with pytest.raises(lib.DGError, match="UNSUPPORTED"):
        q.run(lib)
    q = Layer(2, 20, 17, 128, 128, "e4m3", seed=16)
    with pytest.raises(lib.DGError, match="UNSUPPORTED"):
        q.run(lib)
    # no tokens: nothing to do
    e = dict(x=d["x"][:0], sfx=d["sfx"][:, :0].contiguous(), ids=d["ids"][:0], weights=d["weights"][:0])
    call(y=y[:0], **e)
