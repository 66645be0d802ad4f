"""Cases of the operators around the FP8 GEMMs: the residual addition with its RMS norm and E4M3
output (and its gradient), the top-k router (and its gradient), and a whole mixture-of-experts layer
for a few tokens with E4M3 or E2M1 expert weights.

`run` computes a case either in plain form (elementary torch operations in 32 bits) or, where `own`
is true, through the library's entry points. `exact` is the same definition in 64 bits.

Formats are the library's: E4M3 activations [T, H] with one UE8M0 scale per row per 128 columns packed
four to an int32, [ceil(H / 512), ceil4(T)]; E4M3 weights with one scale per 128 x 128 block; E2M1
weights with one scale per row per 32 columns.
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decoding step: the norm's launch latency (BF16 y for the router, E4M3 for the products)
        {"name": "norm_decode", "op": "norm", "t": 1, "h": 7168, "stream": "bf16", "weight": "bf16", "y": True, "q": True},
        # a long prompt or a training batch: bandwidth
        {"name": "norm_prefill", "op": "norm", "t": 32768, "h": 7168, "stream": "bf16", "weight": "bf16", "y": False, "q": True},
        # gradient of a short ragged batch with an FP32 residual stream
        {"name": "norm_grad_ragged", "op": "norm_grad", "t": 301, "h": 2048, "stream": "f32", "weight": "f32"},
        # gradient of a training batch
        {"name": "norm_grad_batch", "op": "norm_grad", "t": 16384, "h": 7168, "stream": "bf16", "weight": "bf16"},
        # routing of one decoded token
        {"name": "route_decode", "op": "route", "t": 1, "e": 256, "k": 8, "logits": "bf16", "scoring": "softmax", "renorm": True},
        # routing of a training batch, some experts and some whole rows masked
        {"name": "route_batch", "op": "route", "t": 65536, "e": 256, "k": 8, "logits": "f32", "scoring": "softmax", "renorm": True},
        # the router's gradient: sigmoid scores, few experts, an odd count of BF16 rows
        {"name": "route_grad_odd", "op": "route_grad", "t": 4099, "e": 60, "k": 4, "logits": "bf16", "scoring": "sigmoid", "renorm": True},
        # the router's gradient of a training batch, every expert's logit moves
        {"name": "route_grad_batch", "op": "route_grad", "t": 65536, "e": 256, "k": 8, "logits": "f32", "scoring": "softmax", "renorm": False},
        # one decoded token through a large layer: 8 experts' weights are streamed once
        {"name": "moe_fp8_t1", "op": "moe", "t": 1, "e": 32, "k": 8, "h": 7168, "i": 2048, "w": "e4m3", "c": True},
        # the largest batch of the few-token form, every expert in use
        {"name": "moe_fp8_t32", "op": "moe", "t": 32, "e": 64, "k": 8, "h": 7168, "i": 2048, "w": "e4m3", "c": True},
        # a small layer, three tokens, odd sizes: latency
        {"name": "moe_fp4_small", "op": "moe", "t": 3, "e": 8, "k": 2, "h": 1920, "i": 896, "w": "e2m1", "c": False},
        # a served batch with E2M1 weights
        {"name": "moe_fp4_t16", "op": "moe", "t": 16, "e": 32, "k": 8, "h": 7168, "i": 2048, "w": "e2m1", "c": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over the logarithm."""
    while True:
        v = step * max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))
        if lo <= v <= hi and v not in (3 * 512, 3 * 1024):
            return v


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "route", "route_grad", "moe", "moe", "moe"])
    if op in ("norm", "norm_grad"):
        h = _log(rng, 256, 8192, 128)
        case = {"op": op, "t": _log(rng, 1, min(32768, (32768 if op == "norm" else 16384) * 7168 // (2 * h))), "h": h,
                "stream": rng.choice(["bf16", "f32"]), "weight": rng.choice(["bf16", "f32"])}
        if op == "norm":
            case["q"] = rng.random() < 0.8
            case["y"] = not case["q"] or rng.random() < 0.4
        return case
    if op in ("route", "route_grad"):
        e = _log(rng, 4, 512)
        return {"op": op, "t": _log(rng, 1, min(65536, 65536 * 256 // e)), "e": e, "k": rng.randint(1, min(e, 16)),
                "logits": rng.choice(["bf16", "f32"]), "scoring": rng.choice(["softmax", "sigmoid"]),
                "renorm": rng.random() < 0.6}
    e = _log(rng, 2, 64)
    return {"op": "moe", "t": rng.randint(1, 32), "e": e, "k": rng.randint(1, min(8, e)), "h": _log(rng, 512, 7168, 128),
            "i": _log(rng, 128, 2048, 128), "w": rng.choice(["e4m3", "e2m1"]), "c": rng.random() < 0.5}


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


def _exponents(g, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, device="cuda", generator=g, dtype=torch.uint8)


def _pack(bytes_, mn):
    """UE8M0 bytes [..., mn, groups] -> packed words [..., ceil(groups / 4), ceil4(mn)]."""
    *lead, n, groups = bytes_.shape
    out = torch.zeros(*lead, _up(groups, 4), _up4(mn), 4, device="cuda", dtype=torch.uint8)
    padded = torch.zeros(*lead, n, _up4(groups), device="cuda", dtype=torch.uint8)
    padded[..., :groups] = bytes_
    out[..., :mn, :] = padded.unflatten(-1, (-1, 4)).transpose(-3, -2)
    return out.view(torch.int32).squeeze(-1)


def _stream_like(g, t, h, dtype):
    """A residual stream: unit scale, with a few large channels."""
    s = _normal(g, (t, h))
    s *= torch.where(_uniform(g, (h,)) < 0.004, 30.0, 1.0)
    return s.to(dtype)


def _logits(g, case):
    """Router logits; in batches a share of the rows has experts masked out, and a few rows all of them."""
    t, e = case["t"], case["e"]
    x = _normal(g, (t, e), std=1.5)
    if t > 8:
        row = _uniform(g, (t, 1))
        x = torch.where((row < 0.1) & (_uniform(g, (t, e)) < 0.5), -math.inf, x)
        x = torch.where(row < 0.005, -math.inf, x)
    return x.to(DT[case["logits"]])


def prepare(case, seed):
    g = _gen(case, seed)
    s = dict(case)
    op = case["op"]
    if op == "norm":
        t, h = case["t"], case["h"]
        s["x"] = _normal(g, (t, h), torch.bfloat16)
        s["residual"] = _stream_like(g, t, h, DT[case["stream"]])
        s["gamma"] = (1 + _normal(g, (h,), std=0.1)).to(DT[case["weight"]])
        s["out_sum"] = torch.empty_like(s["residual"])
        s["out_rstd"] = torch.empty(t, device="cuda", dtype=torch.float32)
        s["out_y"] = torch.empty(t, h, device="cuda", dtype=torch.bfloat16) if case["y"] else None
        s["out_q"] = torch.empty(t, h, device="cuda", dtype=torch.float8_e4m3fn) if case["q"] else None
        s["out_sf"] = torch.empty(_up(h, 512), _up4(t), device="cuda", dtype=torch.int32) if case["q"] else None
    elif op == "norm_grad":
        t, h = case["t"], case["h"]
        s["dy"] = _normal(g, (t, h), torch.bfloat16)
        s["sum"] = _stream_like(g, t, h, DT[case["stream"]])
        s["dsum"] = _normal(g, (t, h), DT[case["stream"]])
        s["gamma"] = (1 + _normal(g, (h,), std=0.1)).to(DT[case["weight"]])
        s["rstd"] = torch.rsqrt(s["sum"].float().square().mean(-1) + EPS)
        s["out_dx"] = torch.empty(t, h, device="cuda", dtype=torch.bfloat16)
        s["out_dresidual"] = torch.empty_like(s["sum"]) if case["stream"] == "f32" else None
        s["out_dgamma"] = torch.empty(h, device="cuda", dtype=torch.float32)
    elif op == "route":
        s["x"] = _logits(g, case)
        s["out_ids"] = torch.empty(case["t"], case["k"], device="cuda", dtype=torch.int32)
        s["out_weights"] = torch.empty(case["t"], case["k"], device="cuda", dtype=torch.float32)
    elif op == "route_grad":
        s["x"] = _logits(g, case)
        v, i = torch.sort(s["x"], dim=-1, descending=True, stable=True)
        s["ids"] = torch.where(v > -math.inf, i, -1)[:, :case["k"]].int().contiguous()
        s["dweights"] = _normal(g, (case["t"], case["k"]))
        s["out_dx"] = torch.empty_like(s["x"])
    else:
        t, e, k, h, i = (case[n] for n in ("t", "e", "k", "h", "i"))
        # activations as the norm writes them: rows of unit scale
        s["x"] = (_normal(g, (t, h), std=90.0).clamp_(-448, 448)).to(torch.float8_e4m3fn)
        s["x_exp"] = _exponents(g, (t, h // 128), 119, 121)
        s["sfx"] = _pack(s["x_exp"], t)
        for name, n, kk in (("w13", 2 * i, h), ("w2", h, i)):
            if case["w"] == "e4m3":
                # one expert at a time: the bytes of all of them fit, their 32-bit values need not
                w = torch.empty(e, n, kk, device="cuda", dtype=torch.float8_e4m3fn)
                for a in w:
                    a.copy_(_normal(g, (n, kk), std=90.0).clamp_(-448, 448))
                exps = _exponents(g, (e, _up(n, 128), kk // 128), 114, 116)
                s[name], s[name + "_exp"] = w, exps
                s["sf" + name[1:]] = _pack(exps, _up(n, 128))
            else:
                w = torch.randint(0, 256, (e, n, kk // 2), device="cuda", generator=g, dtype=torch.uint8)
                exps = _exponents(g, (e, n, kk // 32), 119, 121)
                s[name], s[name + "_exp"] = w, exps
                s["sf" + name[1:]] = _pack(exps, n)
        score = _uniform(g, (t, e))
        ids = torch.argsort(score, dim=-1)[:, :k].int()
        if t > 2:
            # a share of the slots holds no expert, and one token none at all
            ids = torch.where(_uniform(g, (t, k)) < 0.05, -1, ids)
            ids[t // 2] = -1
        s["ids"] = ids.contiguous()
        s["weights"] = torch.softmax(_normal(g, (t, k)), dim=-1)
        s["addend"] = _normal(g, (t, h), torch.bfloat16) if case["c"] else None
        s["out_y"] = torch.empty(t, h, device="cuda", dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _norm_plain(s):
    t, h = s["t"], s["h"]
    total = s["x"].float() + s["residual"].float()
    rstd = torch.rsqrt(total.square().mean(-1) + EPS)
    y = total * rstd[:, None] * s["gamma"].float()
    out = {"sum": total.to(s["residual"].dtype), "rstd": rstd}
    if s["y"]:
        out["y"] = y.bfloat16()
    if s["q"]:
        # the least power of two that brings the group's largest magnitude to at most 448 = 0.875 * 2^9
        yg = y.view(t, h // 128, 128)
        mant, ex = torch.frexp(yg.abs().amax(-1))
        n = torch.where(mant == 0, 0, ex - 9 + (mant > 0.875)).clamp(-126, 127)
        out["q"] = torch.ldexp(yg, -n[..., None]).to(torch.float8_e4m3fn).view(t, h)
        out["sf"] = _pack((n + 127).to(torch.uint8), t).view(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _norm_grad_plain(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = s["sum"].float() * rstd
    gy = dy * s["gamma"].float()
    d = rstd * (gy - xhat * (gy * xhat).mean(-1, keepdim=True)) + s["dsum"].float()
    out = {"dx": d.bfloat16(), "dgamma": (dy * xhat).sum(0)}
    if s["out_dresidual"] is not None:
        out["dresidual"] = d.to(s["sum"].dtype)
    return out


def _scores(x, scoring):
    """Each expert's score; an expert whose logit is -inf scores 0, and so does a row that has no other."""
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, 1)


def _route_plain(s):
    x, k = s["x"].float(), s["k"]
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)  # equal logits: the lowest index first
    taken = v[:, :k] > -math.inf
    w = torch.where(taken, torch.gather(_scores(x, s["scoring"]), 1, i[:, :k]), 0)
    if s["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1)
    return {"ids": torch.where(taken, i[:, :k], -1).int(), "weights": w}


def _route_grad_plain(s):
    x, ids = s["x"].float(), s["ids"].long()
    taken = ids >= 0
    at = ids.clamp(min=0)
    p = _scores(x, s["scoring"])
    ps = torch.where(taken, torch.gather(p, 1, at), 0)
    dps = torch.where(taken, s["dweights"], 0)
    if s["renorm"]:
        total = ps.sum(-1, keepdim=True)
        total = torch.where(total > 0, total, 1)
        dps = torch.where(taken, (dps - (dps * ps).sum(-1, keepdim=True) / total) / total, 0)
    dp = torch.zeros_like(x).scatter_add_(1, at, dps)
    dx = dp * p * (1 - p) if s["scoring"] == "sigmoid" else p * (dp - (dp * p).sum(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype)}


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device), e.int() - 127)


def _weights_plain(s, name, of):
    """The 32-bit values of the experts `of` (an index, or all): [experts, n, k]."""
    w, e = s[name][of], s[name + "_exp"][of]
    if s["w"] == "e4m3":
        sc = _pow2(e).repeat_interleave(128, dim=1)[:, :w.shape[1]]
        return (w.float().unflatten(-1, (-1, 128)) * sc[..., None]).flatten(-2)
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    value = torch.cat([value, -value])
    both = torch.stack([value[(w & 15).int()], value[(w >> 4).int()]], dim=-1).flatten(-2)
    return (both.unflatten(-1, (-1, 32)) * _pow2(e)[..., None]).flatten(-2)


def _moe_plain(s):
    t, e, k, h, i = (s[n] for n in ("t", "e", "k", "h", "i"))
    x = (s["x"].float().view(t, h // 128, 128) * _pow2(s["x_exp"])[..., None]).view(t, h)
    taken, at = s["ids"] >= 0, s["ids"].clamp(min=0).long()
    if t * k <= e:
        # fewer slots than experts: each slot's weights are taken out
        of, xs = at.flatten(), x.repeat_interleave(k, dim=0)[:, :, None]
        gu = torch.bmm(_weights_plain(s, "w13", of), xs)
        a = gu[:, :i] / (1 + torch.exp(-gu[:, :i])) * gu[:, i:]
        y = torch.bmm(_weights_plain(s, "w2", of), a).view(t, k, h)
        y = torch.where(taken[..., None], y * s["weights"][..., None], 0).sum(1)
    else:
        # every expert on every token, and what is not routed left out of the sum
        gu = torch.matmul(_weights_plain(s, "w13", slice(None)), x.t())
        a = gu[:, :i] / (1 + torch.exp(-gu[:, :i])) * gu[:, i:]
        y = torch.matmul(_weights_plain(s, "w2", slice(None)), a)                      # [e, h, t]
        of = torch.arange(e, device="cuda")[:, None, None]
        coef = torch.where((at[None] == of) & taken[None], s["weights"][None], 0).sum(-1)  # [e, t]
        used = ((at[None] == of) & taken[None]).any(-1)
        y = torch.where(used[:, None], y * coef[:, None], 0).sum(0).t()
    if s["addend"] is not None:
        y = y + s["addend"].float()
    return {"y": y.bfloat16()}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _run_own(s):
    import fp8_gemm_nt_gb300 as dg
    op = s["op"]
    if op == "norm":
        dg.dg_add_rms_norm(s["x"], s["residual"], s["gamma"], EPS, residual_out=s["out_sum"], y=s["out_y"], q=s["out_q"],
                           sf=s["out_sf"], rstd=s["out_rstd"])
        out = {"sum": s["out_sum"], "rstd": s["out_rstd"]}
        if s["y"]:
            out["y"] = s["out_y"]
        if s["q"]:
            out["q"], out["sf"] = s["out_q"], s["out_sf"].view(torch.uint8).view(torch.float8_e8m0fnu)
        return out
    if op == "norm_grad":
        dg.dg_add_rms_norm_backward(s["dy"], s["sum"], s["gamma"], s["rstd"], s["dsum"], s["out_dx"], s["out_dresidual"],
                                    s["out_dgamma"])
        out = {"dx": s["out_dx"], "dgamma": s["out_dgamma"]}
        if s["out_dresidual"] is not None:
            out["dresidual"] = s["out_dresidual"]
        return out
    if op == "route":
        dg.dg_moe_route(s["x"], s["out_ids"], s["out_weights"], scoring=s["scoring"], renormalize=s["renorm"])
        return {"ids": s["out_ids"], "weights": s["out_weights"]}
    if op == "route_grad":
        dg.dg_moe_route_backward(s["x"], s["ids"], s["dweights"], s["out_dx"], scoring=s["scoring"], renormalize=s["renorm"])
        return {"dx": s["out_dx"]}
    layer = dg.dg_moe_fp8_few_tokens if s["w"] == "e4m3" else dg.dg_moe_fp8_fp4_few_tokens
    layer(s["x"], s["sfx"], s["w13"], s["sf13"], s["w2"], s["sf2"], s["ids"], s["weights"], s["addend"], s["out_y"])
    return {"y": s["out_y"]}


def run(state):
    if own:
        return _run_own(state)
    plain = {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "route": _route_plain, "route_grad": _route_grad_plain,
             "moe": _moe_plain}
    return plain[state["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "norm":
        n, st = case["t"] * case["h"], size[case["stream"]]
        b = n * (2 + 2 * st) + case["h"] * size[case["weight"]] + 4 * case["t"]
        b += n * 2 * case["y"] + case["q"] * (n + 4 * _up(case["h"], 512) * _up4(case["t"]))
        return {"bytes": b, "flops": 6 * n}
    if op == "norm_grad":
        n, st = case["t"] * case["h"], size[case["stream"]]
        b = n * (2 + 2 * st + 2 + (st if case["stream"] == "f32" else 0))
        return {"bytes": b + case["h"] * (size[case["weight"]] + 4) + 4 * case["t"], "flops": 12 * n}
    if op == "route":
        return {"bytes": case["t"] * (case["e"] * size[case["logits"]] + 8 * case["k"]), "flops": 4 * case["t"] * case["e"]}
    if op == "route_grad":
        return {"bytes": case["t"] * (2 * case["e"] * size[case["logits"]] + 8 * case["k"]), "flops": 8 * case["t"] * case["e"]}
    t, e, k, h, i = (case[n] for n in ("t", "e", "k", "h", "i"))
    # experts that some slot names, of tokens that each name k different ones at random; slots that hold none aside
    live = t * k if t <= 2 else (t - 1) * k * 0.95
    used = e * (1 - (1 - live / (t * e)) ** t)
    per = 3 * h * i
    wb = per + 3 * _up(h, 128) * _up(i, 128) if case["w"] == "e4m3" else per / 2 + per / 32
    b = used * wb + t * (h + h / 128 + 2 * h * (2 if case["c"] else 1) + 8 * k)
    return {"bytes": b, "flops": 2 * live * per}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = torch.float64
    if op == "norm":
        v = s["x"].to(f).add_(s["residual"].to(f))
        r = 1 / torch.sqrt(torch.einsum("th,th->t", v, v) / case["h"] + EPS)
        out = {"sum": v.clone(), "rstd": r}
        v.mul_(r[:, None]).mul_(s["gamma"].to(f))
        if case["y"]:
            out["y"] = v
        if case["q"]:
            # codes as they are before their rounding; a scale is a whole power of two, whose exponent has no 64-bit value
            groups = v.unflatten(1, (-1, 128))
            n = torch.ceil(torch.log2(torch.linalg.vector_norm(groups, ord=math.inf, dim=-1).clamp_min(2.0 ** -110) / 448))
            out["q"] = (groups * torch.exp2(-n)[..., None]).flatten(1)
            out["sf"] = None
        return out
    if op == "norm_grad":
        h = case["h"]
        v, dy, r = s["sum"].to(f), s["dy"].to(f), s["rstd"].to(f)
        gy = dy * s["gamma"].to(f)
        # d(v r)/dv with r = (mean v^2 + eps)^(-1/2): r gy - v r^3 <gy, v> / h
        inner = torch.einsum("th,th->t", gy, v)
        out = {"dgamma": torch.einsum("th,th,t->h", dy, v, r)}
        d = gy.mul_(r[:, None]).sub_(v.mul_((inner * r ** 3 / h)[:, None])).add_(s["dsum"].to(f))
        out["dx"] = d
        if case["stream"] == "f32":
            out["dresidual"] = d
        return out
    if op in ("route", "route_grad"):
        x = s["x"].to(f)
        none = (x == -math.inf).all(-1, keepdim=True)
        if case["scoring"] == "sigmoid":
            p = torch.sigmoid(x)
        else:
            p = torch.where(none, 0, torch.softmax(torch.where(none, 0, x), -1))
        if op == "route":
            order = torch.argsort(-x, dim=-1, stable=True)[:, :case["k"]]
            w = torch.take_along_dim(p, order, 1).masked_fill(torch.take_along_dim(x, order, 1) == -math.inf, 0)
            if case["renorm"]:
                w = torch.nan_to_num(w / w.sum(-1, keepdim=True), nan=0.0)
            return {"ids": None, "weights": w}
        sel = torch.zeros_like(x)
        dw = torch.zeros_like(x)
        rows = torch.arange(case["t"], device="cuda")[:, None].expand_as(s["ids"])
        good = s["ids"] >= 0
        sel[rows[good], s["ids"][good].long()] = 1
        dw[rows[good], s["ids"][good].long()] = s["dweights"][good].to(f)
        if case["renorm"]:
            q = sel * p
            tot = q.sum(-1, keepdim=True)
            q = torch.where(tot > 0, q / tot, 0)
            lean = dw - (dw * q).sum(-1, keepdim=True)
            dx = q * lean * ((1 - p) if case["scoring"] == "sigmoid" else 1)
        elif case["scoring"] == "sigmoid":
            dx = dw * p * (1 - p)
        else:
            dx = p * dw - p * (p * dw).sum(-1, keepdim=True)
        return {"dx": dx}
    t, e, k, h, i = (case[n] for n in ("t", "e", "k", "h", "i"))

    def scale(b):
        return torch.exp2(b.to(f) - 127)

    def dense(name, a):
        if case["w"] == "e4m3":
            w = s[name][a].to(f)
            sc = torch.kron(scale(s[name + "_exp"][a]), torch.ones(128, 128, device="cuda", dtype=f))
            return w * sc[:w.shape[0]]
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device="cuda", dtype=f)
        w = torch.empty(s[name].shape[1], 2 * s[name].shape[2], device="cuda", dtype=f)
        w[:, 0::2] = table[(s[name][a] % 16).long()]
        w[:, 1::2] = table[torch.div(s[name][a], 16, rounding_mode="floor").long()]
        return w * scale(s[name + "_exp"][a]).repeat_interleave(32, dim=1)

    x = s["x"].to(f) * scale(s["x_exp"]).repeat_interleave(128, dim=1)
    y = torch.zeros(t, h, device="cuda", dtype=f) if s["addend"] is None else s["addend"].to(f)
    for a in range(e):
        tok, slot = torch.nonzero(s["ids"] == a, as_tuple=True)
        if tok.numel() == 0:
            continue
        z = x[tok] @ dense("w13", a).t()
        gate, up = z[:, :i], z[:, i:]
        y.index_add_(0, tok, s["weights"][tok, slot].to(f)[:, None] * ((gate * torch.sigmoid(gate) * up) @ dense("w2", a).t()))
    return {"y": y}
