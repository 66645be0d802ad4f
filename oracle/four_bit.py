"""FP64 CPU oracle of the four-bit operators and of the router's balance loss: quantisation to E2M1 with
UE8M0 scales per 32 columns, the SwiGLU before it and its gradient, the products of two E2M1 operands, the
balance loss with its counts and its gradient. Test infrastructure only, written from the formulas in
include/dg.h's terms; it shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import decode_e2m1, decode_ue8m0, unpack_e2m1, unpack_sf

BLOCK = 32
MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


# --------------------------------------------------------------------------------------
# quantisation
# --------------------------------------------------------------------------------------

def block_scale_codes(y):
    """UE8M0 codes [..., K/32]: the least e in [1, 254] with max|y_b| <= 6 * 2**(e - 127); 127 for a block of
    zeros, 255 for one with a value that is not finite."""
    y = np.asarray(y, np.float64)
    blocks = np.abs(y.reshape(*y.shape[:-1], y.shape[-1] // BLOCK, BLOCK))
    codes = np.empty(blocks.shape[:-1], np.int64)
    for at in np.ndindex(codes.shape):
        b = blocks[at]
        if not np.isfinite(b).all():
            codes[at] = 255
        elif b.max() == 0:
            codes[at] = 127
        else:
            e = max(int(np.floor(np.log2(b.max() / 6))) + 125, 1)        # at or below the answer, then up to it
            while b.max() > np.ldexp(6.0, e - 127):
                e += 1
            codes[at] = e
    return codes


def nearest_e2m1(v):
    """Codes 0..15 of the nearest E2M1 values, of two at the same distance the even code; |v| <= 6."""
    v = np.asarray(v, np.float64)
    gap = np.abs(np.abs(v)[..., None] - MAGNITUDES)
    near = gap == gap.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def quantize_fp4(y):
    """(codes [..., K], scale codes [..., K/32]) of rows y [..., K]."""
    y = np.asarray(y, np.float64)
    e = block_scale_codes(y)
    bad = np.repeat(e == 255, BLOCK, -1)
    v = np.where(bad, 0.0, y) * np.exp2(127.0 - np.repeat(np.minimum(e, 254), BLOCK, -1))
    return np.where(bad, 0, nearest_e2m1(v)).astype(np.uint8), e.astype(np.uint8)


def scale_bytes(sf, rows, K):
    """Packed scale words [..., K/128, ceil4(rows)] -> codes [..., rows, K/32]."""
    sf = np.asarray(sf)
    if sf.ndim == 2:
        return unpack_sf(sf, rows, K // BLOCK)
    return np.stack([scale_bytes(s, rows, K) for s in sf])


def values(packed, sf):
    """Values [..., rows, K] of packed codes [..., rows, K/2] and their scale words."""
    K = 2 * packed.shape[-1]
    s = decode_ue8m0(scale_bytes(sf, packed.shape[-2], K))
    return decode_e2m1(unpack_e2m1(packed, K)) * np.repeat(s, BLOCK, -1)


def values_of(codes, e):
    """Values of codes [..., K] and scale codes [..., K/32]."""
    return decode_e2m1(codes) * np.repeat(decode_ue8m0(e), BLOCK, -1)


def swiglu(x):
    gate, up = np.split(np.asarray(x, np.float64), 2, axis=-1)
    return gate / (1 + np.exp(-gate)) * up


def swiglu_backward(x, dy):
    gate, up = np.split(np.asarray(x, np.float64), 2, axis=-1)
    s = 1 / (1 + np.exp(-gate))
    return np.concatenate([dy * up * s * (1 + gate * (1 - s)), dy * gate * s], -1)


# --------------------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------------------

def gemm(a, sfa, b, sfb, c=None):
    """C + A @ B.T of packed operands [M, K/2] and [N, K/2]."""
    d = values(a, sfa) @ values(b, sfb).T
    return d if c is None else d + np.asarray(c, np.float64)


def gemm_magnitude(a, sfa, b, sfb):
    """The sums of the terms' magnitudes."""
    return np.abs(values(a, sfa)) @ np.abs(values(b, sfb)).T


# --------------------------------------------------------------------------------------
# balance loss
# --------------------------------------------------------------------------------------

def probabilities(logits, scoring):
    """p [T, E]: each row's scores over the experts that are not masked, made to add up to one."""
    p = np.zeros(np.shape(logits))
    for t, row in enumerate(np.asarray(logits, np.float64)):
        live = row > -np.inf
        if live.any():
            z = row[live] if scoring == "softmax" else -np.logaddexp(0, -row[live])
            z = np.exp(z - z.max())
            p[t, live] = z / z.sum()
    return p


def balance_loss(logits, ids, scoring="softmax", coef=1.0):
    """(loss, counts [E], live rows, prob_mean [E])."""
    E = np.shape(logits)[1]
    ids = np.asarray(ids)
    counts = np.array([np.sum(ids == e) for e in range(E)])
    live = int((np.asarray(logits, np.float64) > -np.inf).any(-1).sum())
    mean = probabilities(logits, scoring).sum(0) / max(live, 1)
    return coef * E * np.dot(counts / max(counts.sum(), 1), mean), counts, live, mean


def balance_loss_backward(logits, counts, live, dloss, scoring="softmax", coef=1.0):
    logits = np.asarray(logits, np.float64)
    p = probabilities(logits, scoring)
    f = np.asarray(counts) / max(np.sum(counts), 1)
    d = dloss * coef * logits.shape[1] / max(live, 1) * p * (f - (p @ f)[:, None])
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            d = np.where(p > 0, d / (1 + np.exp(np.where(p > 0, logits, 0))), 0)
    return d
