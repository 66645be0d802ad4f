"""FP64 CPU oracle of the operators around the GEMMs: the residual addition with its RMS norm and
E4M3 output, the top-k router, both gradients, and the mixture-of-experts layer. Test infrastructure
only, written from the formulas in include/dg.h's terms; it shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import decode_e2m1, decode_e4m3, decode_ue8m0, unpack_e2m1, unpack_sf

GROUP = 128


# --------------------------------------------------------------------------------------
# norm
# --------------------------------------------------------------------------------------

def add_rms_norm(x, residual, weight, eps):
    """(s, rstd, y) of rows x [T, H]; residual may be None."""
    s = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=-1) + eps)
    return s, rstd, s * rstd[:, None] * np.asarray(weight, np.float64)


def group_scale_codes(y):
    """UE8M0 codes [T, H/128]: the least e in [1, 254] with max|y_g| <= 448 * 2**(e - 127) over the
    group's finite elements; 127 for a group without a nonzero one."""
    T, H = y.shape
    amax = np.where(np.isfinite(y), np.abs(y), 0.0).reshape(T, H // GROUP, GROUP).max(-1)
    codes = np.empty(amax.shape, np.int64)
    for at, m in np.ndenumerate(amax):
        e = 127
        if m > 0:
            e = int(np.floor(np.log2(m / 448.0))) + 125       # below the answer, then up to it
            while m > np.ldexp(448.0, e - 127):
                e += 1
        codes[at] = min(max(e, 1), 254)
    return codes


def add_rms_norm_backward(dy, s, weight, rstd, ds):
    """(d, dw): gradients of sum(dy * y) + sum(ds * s) with respect to s and to weight, for the rstd of s."""
    dy, s, rstd = (np.asarray(v, np.float64) for v in (dy, s, rstd))
    xhat = s * rstd[:, None]
    g = dy * np.asarray(weight, np.float64)
    d = rstd[:, None] * (g - xhat * np.mean(g * xhat, axis=-1, keepdims=True))
    return d if ds is None else d + np.asarray(ds, np.float64), (dy * xhat).sum(0)


# --------------------------------------------------------------------------------------
# router
# --------------------------------------------------------------------------------------

def _scores(row, scoring):
    """Scores of a row; masked experts (-inf, NaN) score 0."""
    live = row > -np.inf
    p = np.zeros(row.shape)
    if scoring == "sigmoid":
        p[live] = 1.0 / (1.0 + np.exp(-row[live]))
    elif live.any():
        p[live] = np.exp(row[live] - row[live].max())
        p /= p.sum()
    return p


def moe_route(logits, k, scoring="softmax", renormalize=True, scale=1.0):
    """(ids [T, k], weights [T, k])."""
    logits = np.asarray(logits, np.float64)
    ids = np.full((len(logits), k), -1, np.int64)
    w = np.zeros((len(logits), k))
    for t, row in enumerate(logits):
        live = [e for e in range(len(row)) if row[e] > -np.inf]
        chosen = sorted(live, key=lambda e: (-row[e], e))[:k]
        p = _scores(row, scoring)[chosen]
        if renormalize:
            p = p / p.sum() if p.sum() > 0 else np.zeros_like(p)
        ids[t, :len(chosen)], w[t, :len(chosen)] = chosen, scale * p
    return ids, w


def moe_route_backward(logits, ids, dweights, scoring="softmax", renormalize=True, scale=1.0):
    """dlogits [T, E], through the scores p: dw -> dp -> dlogits."""
    logits = np.asarray(logits, np.float64)
    out = np.zeros(logits.shape)
    for t, row in enumerate(logits):
        sel = ids[t] >= 0
        at = ids[t][sel]
        p = _scores(row, scoring)
        d = scale * np.asarray(dweights, np.float64)[t][sel]
        if renormalize:
            total = p[at].sum()
            d = (d - (d * p[at]).sum() / total) / total if total > 0 else np.zeros_like(d)
        dp = np.zeros_like(row)
        dp[at] = d
        if scoring == "sigmoid":
            out[t] = dp * p * (1 - p)
        else:
            out[t] = p * (dp - (dp * p).sum())
    return out


# --------------------------------------------------------------------------------------
# mixture-of-experts layer
# --------------------------------------------------------------------------------------

def expert_matrix(codes, sf, b_format, N, K):
    """One expert's [N, K] values from its codes and packed scales."""
    if b_format == "e4m3":
        s = decode_ue8m0(unpack_sf(sf, -(-N // GROUP), K // GROUP))
        return decode_e4m3(codes) * np.repeat(np.repeat(s, GROUP, 0)[:N], GROUP, 1)
    words = np.ascontiguousarray(sf).view(np.uint8).reshape(K // GROUP, -1, 4)[:, :N]      # [K/128, N, 4]
    s = decode_ue8m0(words.transpose(1, 0, 2).reshape(N, K // 32))
    return decode_e2m1(unpack_e2m1(codes, K)) * np.repeat(s, 32, 1)


def activations(x, sfx, T, H):
    return decode_e4m3(x) * np.repeat(decode_ue8m0(unpack_sf(sfx, T, H // GROUP)), GROUP, 1)


def moe_layer(x, sfx, w13, sf13, w2, sf2, ids, weights, c, b_format="e4m3", bound=None):
    """y [T, H] = c + sum over the slots of weight * w2[e] (silu(gate) * up). `bound`, if given, is a
    dict that receives "y": how far a result may be that rounds the inner products to `bound["dot"]` of
    the sum of their terms' magnitudes and the inner values to `bound["inner"]` of themselves."""
    T, H = x.shape
    I = w2.shape[2] * (2 if b_format == "e2m1" else 1)
    xv = activations(x, sfx, T, H)
    y = np.zeros((T, H)) if c is None else np.asarray(c, np.float64).copy()
    err = np.zeros((T, H))
    for e in sorted({int(v) for v in ids.reshape(-1) if 0 <= v < w13.shape[0]}):
        a13 = expert_matrix(w13[e], sf13[e], b_format, 2 * I, H)
        a2 = expert_matrix(w2[e], sf2[e], b_format, H, I)
        for t in range(T):
            slots = np.nonzero(ids[t] == e)[0]
            if len(slots) == 0:
                continue
            z = a13 @ xv[t]
            gate, up = z[:I], z[I:]
            silu = gate / (1 + np.exp(-gate))
            w = float(np.sum(np.asarray(weights, np.float64)[t, slots]))
            h = w * silu * up
            y[t] += a2 @ h
            if bound is not None:
                dz = bound["dot"] * (np.abs(a13) @ np.abs(xv[t]))
                dh = abs(w) * (1.1 * np.abs(up) * dz[:I] + np.abs(silu) * dz[I:] + 1.1 * dz[:I] * dz[I:]) + bound["inner"] * np.abs(h)
                err[t] += np.abs(a2) @ (dh + bound["dot"] * np.abs(h))
    if bound is not None:
        bound["y"] = err
    return y
