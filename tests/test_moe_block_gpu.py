"""The example that runs the operators together: its output and its router's gradient against 64 bits.

Tolerances, in the Euclidean norm: `out` is rounded to BF16 after s was, each within 2^-8 / sqrt(3) of the
values, and the experts' part is within 2^-10 before: 1.5 * 2^-8 in all. A gradient passes at most eight
roundings to BF16 (dlogits, dn, n, dx or ds, and their sums), each 2^-8 of what it rounds: 2^-5."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import oracle.layers as OL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens, experts, topk, hidden, inner, fp4", [(1, 16, 2, 256, 128, False), (9, 48, 3, 640, 256, True), (32, 16, 4, 512, 384, False)])
def test_block(tokens, experts, topk, hidden, inner, fp4):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block as M

    block = M.MoeBlock(hidden, inner, experts, topk, fp4, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, residual, dout = (torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16() for _ in range(3))
    b = block.buffers(tokens)
    out = block.step(x, residual, b)
    far = lambda got, want: np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)  # noqa: E731
    assert far(out, M.reference(block, x, residual, b)) <= 1.5 * 2.0 ** -8

    logits, ids = b["logits"].double().cpu().numpy(), b["ids"].cpu().numpy()
    want_ids, _ = OL.moe_route(logits, topk)[:2]
    assert (ids == want_ids).all()
    dweights = torch.randn(tokens, topk, device="cuda", generator=g)
    dx, ds, dgamma, drouter = block.router_gradient(b, dweights, dout)
    dlogits = OL.moe_route_backward(logits, ids, dweights.double().cpu().numpy())
    s, gamma = b["s"].double().cpu().numpy(), block.host["gamma"].astype(np.float64)
    rstd = 1 / np.sqrt(np.mean(s * s, -1) + M.EPS)
    n = s * rstd[:, None] * gamma
    want = OL.add_rms_norm_backward(dlogits @ block.router_bf16.double().cpu().numpy(), s, gamma, rstd, dout.double().cpu().numpy())
    for name, got, exact in (("dx", dx, want[0]), ("ds", ds, want[0]), ("dgamma", dgamma, want[1]), ("drouter", drouter, dlogits.T @ n)):
        assert far(got, exact) <= 2.0 ** -5, name
