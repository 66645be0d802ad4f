"""A mixture-of-experts layer in four bits, weights and activations, for any number of tokens, with the balance loss that
trains its router:

    ids, w = top-k of the softmax of logits         dg_moe_route
    loss, counts                                    dg_moe_balance_loss: counts are what the masked products go by
    rows of each expert's tokens, in FP4            dg_quantize_fp4
    z = rows @ w13.T                                dg_m_grouped_fp4_gemm_nt_masked
    h = silu(gate) * up of z, in FP4                dg_swiglu_quantize_fp4
    y = h @ w2.T, out = sum_j w_j y                 dg_m_grouped_fp4_gemm_nt_masked

and gradients: of the logits, through the weights and the balance loss (dg_moe_route_backward,
dg_moe_balance_loss_backward), and of z (dg_swiglu_backward). The gathering of the rows and the weighted sum, for which the
library has no operator, are some ten PyTorch operations, the larger part of an eager step's launches.

    python examples/moe_four_bit.py [--tokens 256] [--experts 32] [--topk 4] [--hidden 2048] [--inner 1024]

prints how far `out` is from the layer computed in 64 bits from the same codes, and the time of a step, eager and as a
CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_gemm_nt_gb300 as dg  # noqa: E402

COEF = 0.01


def quantized(x: torch.Tensor):
    """(codes, scales) of rows [.., M, K]."""
    q = torch.empty(*x.shape[:-1], x.shape[-1] // 2, dtype=torch.uint8, device=x.device)
    sf = torch.empty(*x.shape[:-2], x.shape[-1] // 128, 4 * (-(-x.shape[-2] // 4)), dtype=torch.int32, device=x.device)
    return dg.dg_quantize_fp4(x, q, sf)


class FourBitExperts:
    """Random weights on the current device."""

    def __init__(self, hidden: int, inner: int, experts: int, topk: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.inner, self.experts, self.topk = hidden, inner, experts, topk
        weight = lambda n, k: torch.randn(experts, n, k, device="cuda", generator=g).bfloat16() / k ** 0.5  # noqa: E731
        self.w13, self.sf13 = quantized(weight(2 * inner, hidden))
        self.w2, self.sf2 = quantized(weight(hidden, inner))

    def buffers(self, tokens: int) -> dict:
        """What a step writes; allocated once for a number of tokens. An expert has room for every token."""
        new = lambda dtype, *shape: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
        E, T, H, I = self.experts, tokens, self.hidden, self.inner
        padded = 4 * (-(-T // 4))
        return {"ids": new(torch.int32, T, self.topk), "weights": new(torch.float32, T, self.topk), "counts": new(torch.int32, E),
                "live": new(torch.int32, 1), "probs": new(torch.float32, E), "loss": new(torch.float32, 1),
                "rows": new(torch.bfloat16, E * T + 1, H), "q": new(torch.uint8, E, T, H // 2), "sf": new(torch.int32, E, H // 128, padded),
                "z": new(torch.bfloat16, E, T, 2 * I), "h": new(torch.uint8, E, T, I // 2), "sfh": new(torch.int32, E, I // 128, padded),
                "y": new(torch.bfloat16, E * T + 1, H)}

    def step(self, x: torch.Tensor, logits: torch.Tensor, b: dict) -> torch.Tensor:
        E, T, H = self.experts, len(x), self.hidden
        dg.dg_moe_route(logits, b["ids"], b["weights"])
        dg.dg_moe_balance_loss(logits, b["ids"], b["counts"], b["live"], b["probs"], b["loss"], coef=COEF)
        # each slot's place: its expert's rows in the order of the tokens; empty slots share a row behind the last
        ids = b["ids"].long().flatten()
        chosen = torch.nn.functional.one_hot(torch.where(ids >= 0, ids, E), E + 1)
        place = torch.where(ids >= 0, ids * T + (chosen.cumsum(0) * chosen).sum(-1) - 1, E * T)
        b["place"] = place
        b["rows"][place] = x.repeat_interleave(self.topk, 0)
        dg.dg_quantize_fp4(b["rows"][:-1].view(E, T, H), b["q"], b["sf"], masked_m=b["counts"])
        dg.dg_m_grouped_fp4_gemm_nt_masked(b["q"], b["sf"], self.w13, self.sf13, b["z"], b["counts"])
        dg.dg_swiglu_quantize_fp4(b["z"], b["h"], b["sfh"], masked_m=b["counts"])
        dg.dg_m_grouped_fp4_gemm_nt_masked(b["h"], b["sfh"], self.w2, self.sf2, b["y"][:-1].view(E, T, H), b["counts"])
        return (b["y"][place].view(T, self.topk, H).float() * b["weights"][..., None]).sum(1).bfloat16()

    def router_gradient(self, logits: torch.Tensor, b: dict, dweights: torch.Tensor, dloss: torch.Tensor) -> torch.Tensor:
        """That of the logits, from those of the routing weights [T, k] and of the loss [1]."""
        dlogits = torch.empty_like(logits)
        dg.dg_moe_route_backward(logits, b["ids"], dweights, dlogits)
        return dg.dg_moe_balance_loss_backward(logits, b["counts"], b["live"], dloss, dlogits, base=dlogits, coef=COEF)

    def inner_gradient(self, b: dict, dh: torch.Tensor) -> torch.Tensor:
        """That of z [E, T, 2 I], from that of silu(gate) * up [E, T, I]; rows behind the counts are 0."""
        return dg.dg_swiglu_backward(b["z"], dh, torch.zeros_like(b["z"]), masked_m=b["counts"])


def reference(layer: FourBitExperts, b: dict) -> np.ndarray:
    """out in 64 bits, from the codes of the last step's rows and of the weights."""
    import oracle.four_bit as F

    at = lambda t: t.cpu().numpy()  # noqa: E731
    T, k = b["ids"].shape
    y = np.zeros((layer.experts * T + 1, layer.hidden))
    for e, c in enumerate(b["counts"].tolist()):
        if c:
            z = F.values(at(b["q"][e]), at(b["sf"][e]))[:c] @ F.values(at(layer.w13[e]), at(layer.sf13[e])).T
            h = F.values_of(*F.quantize_fp4(F.swiglu(z)))
            y[e * T:e * T + c] = h @ F.values(at(layer.w2[e]), at(layer.sf2[e])).T
    return (y[at(b["place"])].reshape(T, k, -1) * at(b["weights"]).astype(np.float64)[..., None]).sum(1)


def main() -> None:
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 256), ("experts", 32), ("topk", 4), ("hidden", 2048), ("inner", 1024)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    layer = FourBitExperts(a.hidden, a.inner, a.experts, a.topk)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, logits = torch.randn(a.tokens, a.hidden, device="cuda", generator=g).bfloat16(), torch.randn(a.tokens, a.experts, device="cuda", generator=g)
    b = layer.buffers(a.tokens)
    out = layer.step(x, logits, b)
    want = reference(layer, b)
    print(f"out: {np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want):.2e} of its norm from 64 bits, balance loss {float(b['loss']):.5f}")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer.step(x, logits, b)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            layer.step(x, logits, b)
        for name, run in (("eager", lambda: layer.step(x, logits, b)), ("graph", graph.replay)):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            run()
            begin.record(s)
            for _ in range(50):
                run()
            end.record(s)
            s.synchronize()
            print(f"{name}: {begin.elapsed_time(end) * 20:.1f} us a step")


if __name__ == "__main__":
    main()
