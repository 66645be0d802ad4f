"""Cases of the four-bit operators beside the FP8 GEMMs and the router: quantisation to E2M1 with a
scale per 32 columns, alone and behind the gate of a SwiGLU (with the gate's gradient), the products of
two E2M1 operands (dense, M-grouped contiguous and masked), and the balance loss of a router with its
counts per expert and its gradient.

`run` computes a case either in plain form (elementary torch operations in 32 bits) or, where `own`
is true, through the library's entry points. `exact` is the same definition in 64 bits.

Formats are the library's: E2M1 rows, two codes a byte, the even column in the low nibble: uint8
[(G,) M, K / 2]; one UE8M0 scale per row per 32 columns, packed four to an int32 [(G,) K / 128, ceil4(M)].
"""
import math

import torch

own = False

COEF = 0.01
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the activations of one decoded token: latency
        {"name": "quantize_token", "op": "quantize", "g": 0, "m": 1, "k": 7168, "x": "bf16"},
        # the activations of a long prompt: bandwidth
        {"name": "quantize_prefill", "op": "quantize", "g": 0, "m": 32768, "k": 7168, "x": "bf16"},
        # between the two products of the masked layout: ragged counts, some experts without a token
        {"name": "swiglu_masked", "op": "swiglu", "g": 32, "m": 256, "k": 2048},
        # the gate's gradient of a training batch
        {"name": "swiglu_grad_batch", "op": "swiglu_grad", "g": 0, "m": 8192, "k": 2048},
        # one token through a small layer: latency
        {"name": "gemm_token", "op": "dense", "m": 1, "n": 2048, "k": 1536, "c": False},
        # a decoding batch against one large weight: its bytes are streamed once
        {"name": "gemm_decode", "op": "dense", "m": 128, "n": 7168, "k": 16384, "c": True},
        # a prompt's tokens with a short K: the output's bytes count
        {"name": "gemm_prefill", "op": "dense", "m": 4096, "n": 24576, "k": 1536, "c": False},
        # a training batch over eight experts: arithmetic
        {"name": "gemm_contiguous", "op": "contiguous", "g": 8, "m": 32768, "n": 4096, "k": 7168},
        # a served batch over many experts, counts known to the device alone: the weights' bytes
        {"name": "gemm_masked", "op": "masked", "g": 32, "m": 256, "n": 7168, "k": 2048},
        # the loss of a short batch: an odd count of experts and of BF16 rows, sigmoid scores
        {"name": "balance_odd", "op": "balance", "t": 4099, "e": 60, "k": 4, "logits": "bf16", "scoring": "sigmoid"},
        # the loss of a training batch, some experts and some whole rows masked
        {"name": "balance_batch", "op": "balance", "t": 65536, "e": 256, "k": 8, "logits": "f32", "scoring": "softmax"},
        # its gradient, added to the one of the router's weights
        {"name": "balance_grad_batch", "op": "balance_grad", "t": 65536, "e": 256, "k": 8, "logits": "f32", "scoring": "softmax", "base": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over the logarithm."""
    while True:
        v = step * max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))
        if lo <= v <= hi:
            return v


def draw(rng):
    op = rng.choice(["quantize", "swiglu", "swiglu_grad", "dense", "dense", "dense", "contiguous", "masked", "masked", "balance", "balance_grad"])
    if op == "quantize":
        g, k = rng.choice([0, 0, 3, 32]), _log(rng, 128, 16384, 128)
        return {"op": op, "g": g, "m": _log(rng, 1, min(32768, 32768 * 3584 // (k * max(g, 1)))), "k": k, "x": rng.choice(["bf16", "f32"])}
    if op in ("swiglu", "swiglu_grad"):
        g, k = rng.choice([0, 4, 32]), _log(rng, 128, 4096, 128)
        return {"op": op, "g": g, "m": _log(rng, 1, min(8192, 8192 * 2048 // (k * max(g, 1)))), "k": k}
    if op == "dense":
        n, k = _log(rng, 16, 24576, 16), _log(rng, 128, 16384, 128)
        return {"op": op, "m": _log(rng, 1, 4096), "n": n, "k": k, "c": rng.random() < 0.5}
    if op == "contiguous":
        n, k = _log(rng, 128, 4096, 16), _log(rng, 128, 7168, 128)
        return {"op": op, "g": rng.randint(1, 16), "m": _log(rng, 128, 16384), "n": n, "k": k}
    if op == "masked":
        n, k = _log(rng, 128, 7168, 16), _log(rng, 128, 4096, 128)
        return {"op": op, "g": _log(rng, 1, 48), "m": _log(rng, 1, 300), "n": n, "k": k}
    e = _log(rng, 4, 512)
    case = {"op": op, "t": _log(rng, 1, min(65536, 65536 * 256 // e)), "e": e, "k": rng.randint(1, min(e, 16)),
            "logits": rng.choice(["bf16", "f32"]), "scoring": rng.choice(["softmax", "sigmoid"])}
    if op == "balance_grad":
        case["base"] = rng.random() < 0.6
    return case


def _up(a, b):
    return -(-a // b)


def _up4(a):
    return 4 * _up(a, 4)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + sum(ord(ch) * (i + 1) for i, ch in enumerate(case["op"])))
    return g


def _normal(g, shape, dtype=torch.float32, std=1.0):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0, std, generator=g)


def _uniform(g, shape):
    return torch.rand(shape, device="cuda", generator=g)


def _pack(bytes_):
    """UE8M0 bytes [..., m, groups] -> packed words [..., groups / 4, ceil4(m)]."""
    *lead, m, groups = bytes_.shape
    out = torch.zeros(*lead, groups // 4, _up4(m), 4, device="cuda", dtype=torch.uint8)
    out[..., :m, :] = bytes_.unflatten(-1, (-1, 4)).transpose(-3, -2)
    return out.view(torch.int32).squeeze(-1)


def _stream_like(g, shape, dtype):
    """Activations: rows of unlike scale, and a few large channels."""
    s = _normal(g, shape)
    s *= torch.exp(_normal(g, (*shape[:-1], 1)))
    s *= torch.where(_uniform(g, (shape[-1],)) < 0.004, 20.0, 1.0)
    return s.to(dtype)


def _operand(g, shape):
    """An operand as a quantiser leaves it: packed codes, and the scales' bytes. One group at a time."""
    *lead, rows, k = shape
    q = torch.empty(*lead, rows, k // 2, device="cuda", dtype=torch.uint8)
    e = torch.empty(*lead, rows, k // 32, device="cuda", dtype=torch.uint8)
    for a, b in zip(q.view(-1, rows, k // 2), e.view(-1, rows, k // 32)):
        x = _normal(g, (rows, k)) * torch.exp(0.5 * _normal(g, (rows, 1)))
        codes, exps = _quantize_plain(x)
        a.copy_(_nibbles(codes))
        b.copy_(exps)
    return q, e


def _counts(g, groups, m):
    """Valid rows of each expert; some have none, some all."""
    c = torch.randint(0, m + 1, (groups,), device="cuda", generator=g, dtype=torch.int32)
    if groups > 2:
        c[1], c[2] = 0, m
    return c


def _logits(g, case):
    """Router logits; in batches a share of the rows has experts masked out, and a few rows all of them."""
    t, e = case["t"], case["e"]
    x = _normal(g, (t, e), std=1.5) + 0.5 * _normal(g, (e,))
    if t > 8:
        row = _uniform(g, (t, 1))
        x = torch.where((row < 0.1) & (_uniform(g, (t, e)) < 0.5), -math.inf, x)
        x = torch.where(row < 0.005, -math.inf, x)
    return x.to(DT[case["logits"]])


def prepare(case, seed):
    g = _gen(case, seed)
    s = dict(case)
    op = case["op"]
    if op in ("quantize", "swiglu", "swiglu_grad"):
        m, k = case["m"], case["k"]
        lead = (case["g"],) if case["g"] else ()
        s["counts"] = _counts(g, case["g"], m) if case["g"] else None
        if op == "quantize":
            s["in"] = _stream_like(g, (*lead, m, k), DT[case["x"]])
        else:
            s["in"] = (_stream_like(g, (*lead, m, 2 * k), torch.float32).clamp_(-60, 60)).to(torch.bfloat16)
        if op == "swiglu_grad":
            s["dy"] = _normal(g, (*lead, m, k), torch.bfloat16)
            s["out_dx"] = torch.zeros(*lead, m, 2 * k, device="cuda", dtype=torch.bfloat16)
        else:
            s["out_q"] = torch.zeros(*lead, m, k // 2, device="cuda", dtype=torch.uint8)
            s["out_sf"] = torch.zeros(*lead, k // 128, _up4(m), device="cuda", dtype=torch.int32)
            # both codes of a byte as the E4M3 bytes of their values
            pair = torch.arange(256, device="cuda")
            value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
            value = torch.cat([value, -value]).to(torch.float8_e4m3fn).view(torch.uint8)
            s["values"] = torch.stack([value[pair % 16], value[pair // 16]], -1).view(torch.int16).squeeze(-1)
        return s
    if op == "dense":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_exp"] = _operand(g, (m, k))
        s["b"], s["b_exp"] = _operand(g, (n, k))
        s["addend"] = _normal(g, (m, n), torch.bfloat16, std=math.sqrt(k)) if case["c"] else None
        s["out_d"] = torch.zeros(m, n, device="cuda", dtype=torch.bfloat16)
    elif op == "contiguous":
        groups, n, k = case["g"], case["n"], case["k"]
        # tokens shared out among the experts, every expert's rows padded to a multiple of 128
        cut = torch.sort(torch.randint(0, case["m"] + 1, (groups - 1,), generator=torch.Generator().manual_seed(int(seed)))).values.tolist()
        sizes = [hi - lo for lo, hi in zip([0] + cut, cut + [case["m"]])]
        index = []
        for expert, rows in enumerate(sizes):
            index += [expert] * rows + [-1] * (-rows % 128)
        s["m_indices"] = torch.tensor(index, dtype=torch.int32, device="cuda")
        s["a"], s["a_exp"] = _operand(g, (len(index), k))
        s["b"], s["b_exp"] = _operand(g, (groups, n, k))
        s["out_d"] = torch.zeros(len(index), n, device="cuda", dtype=torch.bfloat16)
    elif op == "masked":
        groups, m, n, k = case["g"], case["m"], case["n"], case["k"]
        s["counts"] = _counts(g, groups, m)
        s["a"], s["a_exp"] = _operand(g, (groups, m, k))
        s["b"], s["b_exp"] = _operand(g, (groups, n, k))
        s["out_d"] = torch.zeros(groups, m, n, device="cuda", dtype=torch.bfloat16)
    if op in ("dense", "contiguous", "masked"):
        s["sfa"], s["sfb"] = _pack(s["a_exp"]), _pack(s["b_exp"])
        return s
    t, e, k = case["t"], case["e"], case["k"]
    s["x"] = _logits(g, case)
    v, i = torch.sort(s["x"], dim=-1, descending=True, stable=True)
    s["ids"] = torch.where(v > -math.inf, i, -1)[:, :k].int().contiguous()
    s["out_counts"] = torch.empty(e, device="cuda", dtype=torch.int32)
    s["out_live"] = torch.empty(1, device="cuda", dtype=torch.int32)
    if op == "balance":
        s["out_probs"] = torch.empty(e, device="cuda", dtype=torch.float32)
        s["out_loss"] = torch.empty(1, device="cuda", dtype=torch.float32)
    else:
        s["counts"] = torch.bincount(s["ids"][s["ids"] >= 0].long(), minlength=e).int()
        s["live"] = (s["x"] > -math.inf).any(-1).sum().int().view(1)
        s["dloss"] = _normal(g, (1,)) + 2
        # a gradient of the size that this one has: 1 / T
        s["add"] = (_normal(g, (t, e)) * (COEF / t)).to(DT[case["logits"]]) if case["base"] else None
        s["out_dx"] = torch.empty_like(s["x"])
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _quantize_plain(x):
    """Codes 0..15 [..., k] and scale bytes [..., k / 32] of 32-bit rows."""
    g = x.unflatten(-1, (-1, 32))
    # the least power of two that brings the largest magnitude to at most 6 = 0.75 * 2^3
    mant, ex = torch.frexp(g.abs().amax(-1))
    n = torch.where(mant == 0, 0, ex - 3 + (mant > 0.75)).clamp(-126, 127)
    v = torch.ldexp(g, -n[..., None])
    a = v.abs()
    # the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; halfway between two, the one with an even code
    code = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    return (code + 8 * torch.signbit(v)).byte().flatten(-2), (n + 127).to(torch.uint8)


def _nibbles(codes):
    pairs = codes.unflatten(-1, (-1, 2))
    return pairs[..., 0] | (pairs[..., 1] << 4)


def _silu_mul(x):
    gate, up = x.float().chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _valid(s, m):
    """Which rows count: [(g,) m, 1]; all where there are no counts."""
    if s["counts"] is None:
        return torch.ones(m, 1, device="cuda", dtype=torch.bool)
    return (torch.arange(m, device="cuda")[None] < s["counts"][:, None])[..., None]


def _codes_out(s, q, sf):
    """The values that the codes and the scales stand for."""
    return {"q": s["values"][q.int()].view(torch.float8_e4m3fn), "sf": sf.view(torch.uint8).view(torch.float8_e8m0fnu)}


def _quantize_run(s):
    x = s["in"].float() if s["op"] == "quantize" else _silu_mul(s["in"])
    codes, exps = _quantize_plain(x)
    valid = _valid(s, s["m"])                       # rows behind the count stay as they were: zeros here
    return _codes_out(s, torch.where(valid, _nibbles(codes), 0), _pack(torch.where(valid, exps, 0)))


def _swiglu_grad_plain(s):
    gate, up = s["in"].float().chunk(2, dim=-1)
    dy = s["dy"].float()
    sig = 1 / (1 + torch.exp(-gate))
    dx = torch.cat([dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig], -1)
    return {"dx": torch.where(_valid(s, s["m"]), dx, 0).bfloat16()}


def _dense_values(s, name):
    """The 32-bit values of an operand: [..., rows, k]."""
    w, e = s[name], s[name + "_exp"]
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    value = torch.cat([value, -value])
    both = torch.stack([value[(w & 15).int()], value[(w >> 4).int()]], dim=-1).flatten(-2)
    return (both.unflatten(-1, (-1, 32)) * torch.ldexp(torch.ones((), device="cuda"), e.int() - 127)[..., None]).flatten(-2)


def _gemm_plain(s):
    a, b = _dense_values(s, "a"), _dense_values(s, "b")
    if s["op"] == "dense":
        y = torch.matmul(a, b.t())
        if s["addend"] is not None:
            y = y + s["addend"].float()
    elif s["op"] == "contiguous":
        # every block of 128 rows with its expert's weights; padding rows stay as they were
        blocks = s["m_indices"].view(-1, 128)
        y = torch.bmm(a.view(-1, 128, s["k"]), b[blocks[:, 0].clamp(min=0).long()].transpose(1, 2)).view(-1, s["n"])
        y = torch.where(s["m_indices"][:, None] >= 0, y, 0)
    else:
        y = torch.where(_valid(s, s["m"]), torch.bmm(a, b.transpose(1, 2)), 0)
    return {"d": y.bfloat16()}


def _probabilities(x, scoring):
    """Each row's scores, made to add up to one; a masked expert has none, and so has a row of nothing else."""
    live = x > -math.inf
    if scoring == "sigmoid":
        p = torch.where(live, 1 / (1 + torch.exp(-x)), 0)
    else:
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(top > -math.inf, top, 0))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, 1)


def _balance_plain(s):
    x, e = s["x"].float(), s["e"]
    ids = s["ids"]
    counts = torch.zeros(e + 1, device="cuda", dtype=torch.int64).scatter_add_(
        0, torch.where(ids >= 0, ids, e).flatten().long(), torch.ones(ids.numel(), device="cuda", dtype=torch.int64))[:e]
    live = (x > -math.inf).any(-1).sum()
    probs = _probabilities(x, s["scoring"]).sum(0) / live.clamp(min=1)
    loss = COEF * e * (counts / counts.sum().clamp(min=1) * probs).sum()
    return {"counts": counts.int(), "live": live.int().view(1), "probs": probs, "loss": loss.view(1)}


def _balance_grad_plain(s):
    x, e = s["x"].float(), s["e"]
    p = _probabilities(x, s["scoring"])
    f = s["counts"] / s["counts"].sum().clamp(min=1)
    dx = s["dloss"] * (COEF * e) / s["live"].clamp(min=1) * p * (f - (p * f).sum(-1, keepdim=True))
    if s["scoring"] == "sigmoid":
        dx = dx / (1 + torch.exp(x))
    dx = torch.where(x > -math.inf, dx, 0)
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return {"dx": dx.to(s["x"].dtype)}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _run_own(s):
    import fp8_gemm_nt_gb300 as dg
    op = s["op"]
    if op == "quantize":
        dg.dg_quantize_fp4(s["in"], s["out_q"], s["out_sf"], masked_m=s["counts"])
        return _codes_out(s, s["out_q"], s["out_sf"])
    if op == "swiglu":
        dg.dg_swiglu_quantize_fp4(s["in"], s["out_q"], s["out_sf"], masked_m=s["counts"])
        return _codes_out(s, s["out_q"], s["out_sf"])
    if op == "swiglu_grad":
        return {"dx": dg.dg_swiglu_backward(s["in"], s["dy"], s["out_dx"], masked_m=s["counts"])}
    if op == "dense":
        return {"d": dg.dg_fp4_gemm_nt(s["a"], s["sfa"], s["b"], s["sfb"], s["addend"], s["out_d"])}
    if op == "contiguous":
        return {"d": dg.dg_m_grouped_fp4_gemm_nt_contiguous(s["a"], s["sfa"], s["b"], s["sfb"], s["out_d"], s["m_indices"])}
    if op == "masked":
        return {"d": dg.dg_m_grouped_fp4_gemm_nt_masked(s["a"], s["sfa"], s["b"], s["sfb"], s["out_d"], s["counts"])}
    if op == "balance":
        dg.dg_moe_balance_loss(s["x"], s["ids"], s["out_counts"], s["out_live"], s["out_probs"], s["out_loss"],
                               scoring=s["scoring"], coef=COEF)
        return {"counts": s["out_counts"], "live": s["out_live"], "probs": s["out_probs"], "loss": s["out_loss"]}
    return {"dx": dg.dg_moe_balance_loss_backward(s["x"], s["counts"], s["live"], s["dloss"], s["out_dx"], base=s["add"],
                                                  scoring=s["scoring"], coef=COEF)}


def run(state):
    if own:
        return _run_own(state)
    plain = {"quantize": _quantize_run, "swiglu": _quantize_run, "swiglu_grad": _swiglu_grad_plain, "dense": _gemm_plain,
             "contiguous": _gemm_plain, "masked": _gemm_plain, "balance": _balance_plain, "balance_grad": _balance_grad_plain}
    return plain[state["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("quantize", "swiglu", "swiglu_grad"):
        # with counts, half of the rows at random
        n = (case["g"] * case["m"] / 2 if case["g"] else case["m"]) * case["k"]
        if op == "swiglu_grad":
            return {"bytes": 10 * n, "flops": 12 * n}
        per = size[case["x"]] if op == "quantize" else 4
        return {"bytes": n * (per + 1 / 2 + 1 / 32), "flops": (4 if op == "quantize" else 9) * n}
    if op in ("dense", "contiguous", "masked"):
        n, k, groups = case["n"], case["k"], case.get("g", 1)
        m = groups * case["m"] / 2 if op == "masked" else case["m"]
        b = (m + groups * n) * (k / 2 + k / 32) + 2 * m * n * (2 if case.get("c") else 1)
        return {"bytes": b, "flops": 2 * m * n * k}
    t, e = case["t"], case["e"]
    if op == "balance":
        return {"bytes": t * (e * size[case["logits"]] + 4 * case["k"]) + 8 * e + 8, "flops": 4 * t * e}
    return {"bytes": t * e * size[case["logits"]] * (3 if case["base"] else 2) + 4 * e + 8, "flops": 8 * t * e}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = torch.float64
    counts = s.get("counts")

    def kept(v):
        """Rows behind an expert's count: zeros, as prepared."""
        if op == "balance_grad" or counts is None:
            return v
        for a, c in enumerate(counts.tolist()):
            v[a, c:] = 0
        return v

    if op in ("quantize", "swiglu"):
        x = s["in"].to(f)
        if op == "swiglu":
            k = case["k"]
            x = x[..., :k] * torch.sigmoid(x[..., :k]) * x[..., k:]
        groups = x.unflatten(-1, (-1, 32))
        peak = torch.linalg.vector_norm(groups, ord=math.inf, dim=-1)
        # (a logarithm of a whole power of two may be a last bit above it)
        v = groups * torch.exp2(-torch.ceil(torch.log2(peak.clamp_min(2.0 ** -120) / 6) - 2.0 ** -40))[..., None]
        # E2M1's steps are 1/2 below 2, 1 below 4 and 2 above; a scale is a whole power of two, whose exponent has no 64-bit value
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
        return {"q": kept((torch.round(v / step) * step).flatten(-2)), "sf": None}
    if op == "swiglu_grad":
        k = case["k"]
        gate, up, dy = s["in"][..., :k].to(f), s["in"][..., k:].to(f), s["dy"].to(f)
        sig = torch.sigmoid(gate)
        # d(gate sig)/d gate = sig + gate sig (1 - sig)
        return {"dx": kept(torch.cat([(sig + gate * sig * torch.sigmoid(-gate)) * up * dy, gate * sig * dy], -1))}
    if op in ("dense", "contiguous", "masked"):
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda", dtype=f)

        def values(codes, exps):
            v = torch.empty(codes.shape[0], 2 * codes.shape[1], device="cuda", dtype=f)
            v[:, 0::2] = table[(codes % 16).long()]
            v[:, 1::2] = table[torch.div(codes, 16, rounding_mode="floor").long()]
            return v * torch.exp2(exps.to(f) - 127).repeat_interleave(32, dim=1)

        if op == "dense":
            d = values(s["a"], s["a_exp"]) @ values(s["b"], s["b_exp"]).t()
            return {"d": d if s["addend"] is None else d + s["addend"].to(f)}
        d = torch.zeros(s["out_d"].shape, device="cuda", dtype=f)
        for a in range(case["g"]):
            if op == "masked":
                c = int(counts[a])
                d[a, :c] = values(s["a"][a, :c], s["a_exp"][a, :c]) @ values(s["b"][a], s["b_exp"][a]).t()
            else:
                rows = torch.nonzero(s["m_indices"] == a).flatten()
                d[rows] = values(s["a"][rows], s["a_exp"][rows]) @ values(s["b"][a], s["b_exp"][a]).t()
        return {"d": d}
    x, e = s["x"].to(f), case["e"]
    masked = x == -math.inf
    # the logarithms of the scores, whose softmax the probabilities are
    z = (torch.nn.functional.logsigmoid(x) if case["scoring"] == "sigmoid" else x).masked_fill(masked, -math.inf)
    dead = masked.all(-1, keepdim=True)
    p = torch.where(dead, 0, torch.softmax(torch.where(dead, 0, z), -1))
    n = int((~dead).sum())
    if op == "balance":
        c = torch.stack([(s["ids"] == a).sum() for a in range(e)]).to(f)
        probs = p.sum(0) / max(n, 1)
        return {"counts": None, "live": None, "probs": probs, "loss": (COEF * e * torch.dot(c / max(float(c.sum()), 1), probs)).view(1)}
    c = counts.to(f) / max(int(counts.sum()), 1)
    dx = p * c - p * (p @ c)[:, None]
    if case["scoring"] == "sigmoid":
        dx = dx * torch.sigmoid(-x)
    dx = (dx * (float(s["dloss"]) * COEF * e / max(n, 1))).masked_fill(masked, 0)
    return {"dx": dx if s["add"] is None else dx + s["add"].to(f)}
