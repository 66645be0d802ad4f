"""The example that runs the four-bit operators together: each step of it against 64 bits from what the step before left,
the gradients, and the whole of it as a CUDA graph with new inputs.

z and y are sums of K terms, off by (K / 64) 2^-22 of the terms' magnitudes, and rounded to BF16 (2^-8). The gradient of the
logits is the sum of two, the first rounded to FP32 (2^-17 of the router's, 2^-15 of the balance loss's terms)."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import oracle as O
import oracle.four_bit as F
import oracle.layers as OL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_four_bit
    return moe_four_bit


def np64(t):
    return t.double().cpu().numpy()


def inputs(tokens, hidden, experts, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(tokens, experts, device="cuda", generator=g)
    if tokens > 2:
        logits[1] = -float("inf")                    # a padded token: no expert takes it
    return torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16(), logits


def check_product(got, q, sf, w, sfw, count):
    a, b = F.values(q, sf)[:count], F.values(w, sfw)
    want = a @ b.T
    assert (np.abs(got[:count] - want) <= 2.0 ** -8 * np.abs(want) + (a.shape[1] // 64 + 1) * 2.0 ** -22 * (np.abs(a) @ np.abs(b).T)).all()


@pytest.mark.parametrize("tokens, experts, topk, hidden, inner", [(1, 8, 2, 256, 128), (37, 16, 3, 640, 256), (300, 8, 2, 512, 384)])
def test_layer(M, tokens, experts, topk, hidden, inner):
    layer = M.FourBitExperts(hidden, inner, experts, topk, seed=tokens)
    x, logits = inputs(tokens, hidden, experts, tokens)
    b = layer.buffers(tokens)
    out = layer.step(x, logits, b)
    assert M.dg.dg_get_device_status() == 0

    l64 = np64(logits)
    ids, weights = OL.moe_route(l64, topk)
    assert (b["ids"].cpu().numpy() == ids).all()
    loss, counts, live, _ = F.balance_loss(l64, ids, coef=M.COEF)
    assert (b["counts"].cpu().numpy() == counts).all() and int(b["live"]) == live
    assert abs(float(b["loss"]) - loss) <= 2.0 ** -14 * loss
    h = {name: b[name].cpu().numpy() for name in ("q", "sf", "h", "sfh")}
    w = {name: getattr(layer, name).cpu().numpy() for name in ("w13", "sf13", "w2", "sf2")}
    z, y = np64(b["z"]), np64(b["y"])[:-1].reshape(experts, tokens, hidden)
    for e, c in enumerate(counts):
        mine = x[torch.from_numpy((ids == e).any(-1)).cuda()]
        codes, exps = F.quantize_fp4(np64(mine))
        assert (O.unpack_e2m1(h["q"][e][:c], hidden) == codes).all() and (F.scale_bytes(h["sf"][e], tokens, hidden)[:c] == exps).all()
        check_product(z[e], h["q"][e], h["sf"][e], w["w13"][e], w["sf13"][e], c)
        # a step of FP4 is at most a third of a value (and a quarter of the least magnitude of its block's scale)
        v = F.swiglu(z[e][:c])
        scale = O.decode_ue8m0(F.scale_bytes(h["sfh"][e], tokens, inner)[:c])
        assert (np.abs(F.values(h["h"][e], h["sfh"][e])[:c] - v) <= np.maximum(np.abs(v) / 5, np.repeat(scale, 32, -1) / 4) * 1.001).all()
        check_product(y[e], h["h"][e], h["sfh"][e], w["w2"][e], w["sf2"][e], c)
    place, wt = b["place"].cpu().numpy(), np64(b["weights"])
    want = (np.concatenate([y.reshape(-1, hidden), np.zeros((1, hidden))])[place].reshape(tokens, topk, hidden) * wt[..., None])
    assert (np.abs(np64(out) - want.sum(1)) <= 2.0 ** -8 * np.abs(want.sum(1)) + 2.0 ** -20 * np.abs(want).sum(1)).all()

    # gradients
    g = torch.Generator(device="cuda").manual_seed(3)
    dweights, dloss = torch.randn(tokens, topk, device="cuda", generator=g), torch.tensor([0.7], device="cuda")
    got = np64(layer.router_gradient(logits, b, dweights, dloss))
    routed = OL.moe_route_backward(l64, ids, np64(dweights))
    balance = F.balance_loss_backward(l64, counts, live, float(dloss), coef=M.COEF)
    p, f = F.probabilities(l64, "softmax"), counts / max(counts.sum(), 1)
    room = 2.0 ** -15 * 0.7 * M.COEF * experts / max(live, 1) * p * (f + (p @ f)[:, None])
    q = np.zeros_like(l64)                             # the router's own terms: q d and q sum q d
    for t in range(tokens):
        for j in range(topk):
            if ids[t, j] >= 0:
                q[t, ids[t, j]] = weights[t, j] * (abs(float(dweights[t, j])) + np.abs(weights[t] * np64(dweights)[t]).sum())
    assert (np.abs(got - routed - balance) <= 2.0 ** -16 * q + room + 2.0 ** -23 * np.abs(routed + balance)).all()
    dh = torch.randn(experts, tokens, inner, device="cuda", generator=g).bfloat16()
    dz = np64(layer.inner_gradient(b, dh))
    for e, c in enumerate(counts):
        gate, up = np.split(z[e][:c], 2, -1)
        s, d = 1 / (1 + np.exp(-gate)), np64(dh)[e][:c]
        room = np.concatenate([np.abs(d * up * s) * (1 + np.abs(gate)), np.abs(d * gate * s)], -1) * 2.0 ** -17
        want = F.swiglu_backward(z[e][:c], d)
        assert (np.abs(dz[e][:c] - want) <= room + 2.0 ** -8 * np.abs(want)).all() and (dz[e][c:] == 0).all()


def test_as_a_graph_with_new_inputs(M):
    tokens, experts, topk, hidden, inner = 50, 16, 2, 256, 128
    layer = M.FourBitExperts(hidden, inner, experts, topk)
    x, logits = inputs(tokens, hidden, experts, 1)
    b = layer.buffers(tokens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.step(x, logits, b)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = layer.step(x, logits, b)
        for seed in (1, 2, 3):
            nx, nl = inputs(tokens, hidden, experts, seed)
            x.copy_(nx)
            logits.copy_(nl)
            g.replay()
            s.synchronize()
            got, loss = out.clone(), b["loss"].clone()
            other = layer.buffers(tokens)
            assert torch.equal(got, layer.step(nx, nl, other)) and torch.equal(loss, other["loss"])
            s.synchronize()
    assert M.dg.dg_get_device_status() == 0
