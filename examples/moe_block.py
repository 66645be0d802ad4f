"""A mixture-of-experts block of a decoder, for the few tokens of a decoding step, and its router's gradient:

    s      = x + residual                      one call: the sum, its RMS norm in BF16, and the norm in
    n      = rms_norm(s) * gamma               E4M3 with a scale per 128 columns, as the GEMMs take it
    logits = n @ router.T                      dg_fp8_gemm_nt (a multiple of 16 experts)
    ids, w = top-k of the softmax of logits    dg_moe_route
    out    = s + sum_j w_j expert_{ids_j}(n)   dg_moe_fp8_few_tokens / dg_moe_fp8_fp4_few_tokens

    python examples/moe_block.py [--tokens 8] [--experts 32] [--topk 6] [--hidden 1024] [--inner 512] [--fp4]

prints how far `out` is from the block computed in 64 bits, and the time of a step, eager and as a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_gemm_nt_gb300 as dg  # noqa: E402
import workloads as W  # noqa: E402

EPS = 1e-6


def _packed_rows(exps: np.ndarray) -> np.ndarray:
    """Scale exponents [N, K/32] of E2M1 rows -> words [K/128, ceil4(N)]."""
    N, blocks = exps.shape
    out = np.zeros((blocks // 4, W.ceil4(N), 4), np.uint8)
    out[:, :N] = exps.reshape(N, blocks // 4, 4).transpose(1, 0, 2)
    return out.reshape(blocks // 4, -1).view(np.int32)


class MoeBlock:
    """Random weights on the current device, `host` the arrays that they were made from."""

    def __init__(self, hidden: int, inner: int, experts: int, topk: int, fp4: bool = False, seed: int = 0):
        rng = np.random.default_rng(seed)
        self.hidden, self.experts, self.topk, self.fp4 = hidden, experts, topk, fp4

        def weight(rows, cols):
            v = rng.normal(size=(rows, cols)).astype(np.float32) / np.sqrt(cols)
            if fp4:
                codes, exps = W.quantize_fp4_rows(v)
                return codes, _packed_rows(exps)
            codes, exps = W.quantize_blocks(v)
            return codes, W.pack_sf(exps)

        router, router_exps = W.quantize_blocks(rng.normal(size=(experts, hidden)).astype(np.float32) * 3 / np.sqrt(hidden))
        self.host = {"gamma": (1 + 0.1 * rng.normal(size=hidden)).astype(np.float32), "router": router, "router_sf": W.pack_sf(router_exps)}
        for name, rows, cols in (("w13", 2 * inner, hidden), ("w2", hidden, inner)):
            pairs = [weight(rows, cols) for _ in range(experts)]
            self.host[name], self.host[name + "_sf"] = (np.stack(p) for p in zip(*pairs))
        for name, value in self.host.items():
            setattr(self, name, torch.from_numpy(np.ascontiguousarray(value)).cuda())
        blocks = torch.from_numpy(router_exps.astype(np.float32)).cuda()
        scale = torch.exp2(blocks - 127).repeat_interleave(128, 0)[:experts].repeat_interleave(128, 1)
        self.router_bf16 = (self.router.view(torch.float8_e4m3fn).float() * scale).bfloat16()     # for its gradient

    def buffers(self, tokens: int) -> dict:
        """What a step writes; allocated once for a number of tokens."""
        new = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
        rows = (tokens, self.hidden)
        return {"s": new(torch.bfloat16, *rows), "q": new(torch.uint8, *rows), "rstd": new(torch.float32, tokens),
                "sf": new(torch.int32, W.ceil_div(self.hidden, 512), W.ceil4(tokens)), "logits": new(torch.bfloat16, tokens, self.experts),
                "ids": new(torch.int32, tokens, self.topk), "weights": new(torch.float32, tokens, self.topk), "out": new(torch.bfloat16, *rows)}

    def step(self, x: torch.Tensor, residual: torch.Tensor, b: dict) -> torch.Tensor:
        dg.dg_add_rms_norm(x, residual, self.gamma, EPS, residual_out=b["s"], q=b["q"], sf=b["sf"], rstd=b["rstd"])
        dg.dg_fp8_gemm_nt(b["q"], b["sf"], self.router, self.router_sf, None, b["logits"])
        dg.dg_moe_route(b["logits"], b["ids"], b["weights"])
        experts = dg.dg_moe_fp8_fp4_few_tokens if self.fp4 else dg.dg_moe_fp8_few_tokens
        return experts(b["q"], b["sf"], self.w13, self.w13_sf, self.w2, self.w2_sf, b["ids"], b["weights"], b["s"], b["out"])

    def router_gradient(self, b: dict, dweights: torch.Tensor, dout: torch.Tensor):
        """From the gradients of the routing weights [T, k] and of `out` (which passes on to s): those of x and of
        the residual (BF16), of gamma and of the router's weights."""
        dlogits, dx, ds = torch.empty_like(b["logits"]), torch.empty_like(b["s"]), torch.empty_like(b["s"])
        dgamma = torch.empty(self.hidden, dtype=torch.float32, device="cuda")
        dg.dg_moe_route_backward(b["logits"], b["ids"], dweights, dlogits)
        dn = dlogits @ self.router_bf16
        n = (b["s"].float() * b["rstd"][:, None] * self.gamma).bfloat16()
        dg.dg_add_rms_norm_backward(dn, b["s"], self.gamma, b["rstd"], dout, dx, ds, dgamma)
        return dx, ds, dgamma, dlogits.T @ n


def reference(block: MoeBlock, x: torch.Tensor, residual: torch.Tensor, b: dict) -> np.ndarray:
    """`out` in 64 bits, from the step's own E4M3 rows and its choice of experts."""
    import oracle.layers as O
    get = lambda name: b[name].cpu().numpy()  # noqa: E731
    s, _, _ = O.add_rms_norm(x.double().cpu().numpy(), residual.double().cpu().numpy(), block.host["gamma"], EPS)
    h = block.host
    return O.moe_layer(get("q"), get("sf"), h["w13"], h["w13_sf"], h["w2"], h["w2_sf"], get("ids"), get("weights"), s,
                       "e2m1" if block.fp4 else "e4m3")


def _us(call, n: int = 200) -> float:
    for _ in range(20):
        call()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(n):
        call()
    end.record()
    torch.cuda.synchronize()
    return begin.elapsed_time(end) / n * 1e3


def main() -> None:
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 8), ("experts", 32), ("topk", 6), ("hidden", 1024), ("inner", 512)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--fp4", action="store_true", help="experts' weights in E2M1")
    a = p.parse_args()
    block = MoeBlock(a.hidden, a.inner, a.experts, a.topk, a.fp4)
    x, residual = (torch.randn(a.tokens, a.hidden, device="cuda").bfloat16() for _ in range(2))
    b = block.buffers(a.tokens)
    out = block.step(x, residual, b)
    want = reference(block, x, residual, b)
    error = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want)
    grads = block.router_gradient(b, torch.randn(a.tokens, a.topk, device="cuda"), torch.randn_like(out))
    assert all(torch.isfinite(g.float()).all() for g in grads)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        block.step(x, residual, b)                    # creates the stream's workspace
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            block.step(x, residual, b)
        eager, replay = _us(lambda: block.step(x, residual, b)), _us(graph.replay)
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner} in {'E2M1' if a.fp4 else 'E4M3'}, {a.topk} each: "
          f"error {error:.1e} of the output, a step {eager:.1f} us eager, {replay:.1f} us as a graph")


if __name__ == "__main__":
    main()
