"""The inner values of the few-token layer as sums of E4M3 terms, restated in numpy, and a check of the layer that shows
their last bits.

A value h of a block of 64 is held as t1 + t2 / 16 + t3 / 16^2 + t4 / 16^3 times the block's scale, the least power of two
with max|h| at most 448 of it: t1 is h rounded to E4M3, the others what is left, times 16 each time. E4M3 rounds a value
to within 2^-4 of itself, or 2^-10 below 2^-6. So the error is at most 2^-16 of h or 2^-10 / 16^3 = 2^-22 of the scale,
whichever is more, and the largest of the 64 is above 224 scales: 2^-22 / 224 = 2^-29.8 of it.

The check cancels the leading bits: with c = -bf16(P), P the experts' part, y holds P - bf16(P), about 2^-9 of P, to 8
bits of that. How far y may be, as a share of |P|, in norms over the outputs, whose terms' signs are mixed:
  - its own rounding: that of the exact output (about 2^-18.5), and half of that again where y lies near a tie;
  - the terms: each of the four roundings leaves at most 2^-4, 2^-4 / sqrt(3) in the mean, of what it rounds: 2^-19;
  - FP32 sums: chains of H / 32 and I / 32 additions of partial sums that grow to the whole, within 2^-24 each of half
    of it in the mean: (H + I) / 64 * 2^-24."""
from __future__ import annotations

import numpy as np
import torch

import oracle.layers as OL
import workloads as W

BLOCK = 64
TERMS = (1.0, 16.0, 256.0, 4096.0)      # what each term is divided by


def e4m3(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.float8_e4m3fn).double().numpy()


def bf16(v):
    return (W.to_bf16_bits(np.asarray(v, np.float32)).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def scale_of(h):
    """The scale of each block of 64 along the last axis (never below 2^-114, where the last term's code would leave its range)."""
    top = np.abs(h).reshape(*h.shape[:-1], -1, BLOCK).max(-1)
    e = np.ceil(np.log2(np.maximum(top, 2.0 ** -200) / 448.0))
    return np.repeat(np.exp2(np.maximum(e, -114)), BLOCK, -1)


def as_terms(h, steps=TERMS):
    """h as its terms add up (the remainder is scaled by 16 each time, whatever the steps are)."""
    scale = scale_of(h)
    left, total = h / scale, np.zeros(h.shape)
    for s in steps:
        t = e4m3(left)
        total += t / s
        left = (left - t) * 16.0
    return total * scale


def layer(p, inner=lambda h: h):
    """The experts' part of layer `p` (the tests' Layer) in 64 bits, its inner values passed through `inner`."""
    x = OL.activations(p.x, p.sfx, p.T, p.H)
    y = np.zeros((p.T, p.H))
    for e in range(p.E):
        tokens = [t for t in range(p.T) if (p.ids[t] == e).any()]
        if not tokens:
            continue
        w = np.array([p.weights[t][p.ids[t] == e].astype(np.float64).sum() for t in tokens])
        z = x[tokens] @ OL.expert_matrix(p.w13[e], p.sf13[e], p.fmt, 2 * p.I, p.H).T
        gate, up = z[:, :p.I], z[:, p.I:]
        with np.errstate(over="ignore"):
            h = w[:, None] * gate / (1 + np.exp(-gate)) * up
        y[tokens] += inner(h) @ OL.expert_matrix(p.w2[e], p.sf2[e], p.fmt, p.H, p.I).T
    return y


def cancel(p):
    """Gives layer `p` the addend that cancels its experts' part, and returns that part and the exact output."""
    part = layer(p)
    p.c = W.to_bf16_bits((-part).astype(np.float32))
    return part, part + bf16(-part)


def far(got, part, want):
    """How far an output is from the exact one, as a share of the experts' part."""
    return np.linalg.norm(got - want) / np.linalg.norm(part)


def tolerance(p, part, want):
    return 1.5 * far(bf16(want), part, want) + 2.0 ** -19 + (p.H + p.I) / 64 * 2.0 ** -24
