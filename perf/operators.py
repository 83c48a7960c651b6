"""The measured calls of the layer operators around the experts: routing
(moe_route), the dense product with its epilogue (moe_linear), the combine's
gradient (moe_scale_backward) and the gradients of the first two.

Each case is one call as a user's program makes it.  With ``own`` false the
operators are computed in plain torch operations, in 32 bits (64 where a
choice between near values hangs on it); with ``own`` true by the library's
entry points.  ``exact`` computes the same from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 tokens over 128 experts: latency of a short call
        {"name": "route_decode", "op": "route", "tokens": 64, "experts": 128, "top_k": 8, "dtype": "bf16",
         "score": "softmax", "renorm": True, "bias": False, "groups": 1, "keep": 1, "top2": False, "scale": 1.0,
         "masked": 0.0},
        # a ragged batch over an expert count that is no power of two, some experts masked out, full-softmax weights
        {"name": "route_ragged", "op": "route", "tokens": 4999, "experts": 60, "top_k": 6, "dtype": "f16",
         "score": "softmax", "renorm": False, "bias": False, "groups": 1, "keep": 1, "top2": False, "scale": 1.0,
         "masked": 0.1},
        # a long prefill with balance bias and grouped experts
        {"name": "route_prefill", "op": "route", "tokens": 32768, "experts": 256, "top_k": 8, "dtype": "f32",
         "score": "sigmoid", "renorm": True, "bias": True, "groups": 8, "keep": 4, "top2": True, "scale": 2.5,
         "masked": 0.0},
        # the gradient of a short batch's full-softmax weights over 8 experts
        {"name": "route_back_small", "op": "route_back", "tokens": 256, "experts": 8, "top_k": 2, "dtype": "f32",
         "score": "softmax", "renorm": False, "scale": 1.0, "masked": 0.0},
        # the same for a training batch of renormalised sigmoid weights
        {"name": "route_back_train", "op": "route_back", "tokens": 32768, "experts": 256, "top_k": 8, "dtype": "f32",
         "score": "sigmoid", "renorm": True, "scale": 2.5, "masked": 0.0},
        # the combine's gradient for a decode-size batch (fine-tuning on short pieces)
        {"name": "scale_back_small", "op": "scale_back", "tokens": 64, "hidden": 2048, "top_k": 8},
        # ... and for a training batch of wide rows
        {"name": "scale_back_train", "op": "scale_back", "tokens": 4097, "hidden": 7168, "top_k": 8},
        # a shared expert's down projection of one token, added to the routed output
        {"name": "linear_token", "op": "linear", "rows": 1, "cols": 7168, "depth": 2048, "dtype": "bf16",
         "out": "bf16", "act": "none", "bias": False, "residual": True, "pre": False},
        # router logits of a prefill, in 32 bits
        {"name": "linear_router", "op": "linear", "rows": 8192, "cols": 256, "depth": 7168, "dtype": "bf16",
         "out": "f32", "act": "none", "bias": False, "residual": False, "pre": False},
        # a shared expert's gated up projection in training: the pre-activation is kept
        {"name": "linear_swiglu", "op": "linear", "rows": 8192, "cols": 2048, "depth": 7168, "dtype": "bf16",
         "out": "bf16", "act": "swiglu", "bias": False, "residual": False, "pre": True},
        # the router product's gradients from 32-bit logit gradients
        {"name": "linear_back_router", "op": "linear_back", "rows": 8192, "cols": 256, "depth": 7168, "dtype": "bf16",
         "out": "f32", "act": "none", "bias": False},
        # the gated up projection's gradients
        {"name": "linear_back_swiglu", "op": "linear_back", "rows": 8192, "cols": 2048, "depth": 7168,
         "dtype": "bf16", "out": "bf16", "act": "swiglu", "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_back", "scale_back", "linear", "linear", "linear_back"])
    if op in ("route", "route_back"):
        tokens = _log(rng, 1, 32768)
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        experts = max(groups * 2, _log(rng, 4, 256) // groups * groups)
        keep = rng.randint(1, groups)
        c = {"op": op, "tokens": tokens, "experts": experts,
             "top_k": rng.randint(1, min(8, keep * (experts // groups))),
             "dtype": rng.choice(["bf16", "f16", "f32"]), "score": rng.choice(["softmax", "sigmoid"]),
             "renorm": rng.random() < 0.6}
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, keep=keep, top2=rng.random() < 0.5)
        c.update(scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.0, 0.1]))
        return c
    if op == "scale_back":
        return {"op": op, "tokens": _log(rng, 1, 4097), "hidden": 256 * rng.randint(1, 28), "top_k": rng.randint(1, 8)}
    back = op == "linear_back"
    act = rng.choice(_ACTS)
    rows, cols, depth = _log(rng, 1, 8192), _log(rng, 8, 4096), 8 * _log(rng, 8, 896)
    if act == "swiglu":
        cols = (cols + 1) // 2
    dtype = rng.choice(["bf16", "bf16", "f16"])
    c = {"op": op, "rows": rows, "cols": cols, "depth": depth, "dtype": dtype, "out": rng.choice([dtype, dtype, "f32"]),
         "act": act, "bias": rng.random() < 0.5}
    if not back:
        c.update(residual=rng.random() < 0.5, pre=act != "none" and rng.random() < 0.5)
    return c


# --- inputs ------------------------------------------------------------------

def _logits(case, gen):
    """Router logits: unit variance and a spread between tokens, as a trained
    router gives; some experts (and some whole rows) at -inf where asked."""
    T, E = case["tokens"], case["experts"]
    z = torch.randn(T, E, generator=gen, device="cuda") * 1.5
    z += 0.5 * torch.randn(1, E, generator=gen, device="cuda")
    if case["masked"] > 0:
        out = torch.rand(T, E, generator=gen, device="cuda") < case["masked"]
        out |= torch.rand(T, 1, generator=gen, device="cuda") < 0.01
        z = z.masked_fill(out, -math.inf)
    return z.to(_TYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op in ("route", "route_back"):
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        s["logits"] = _logits(case, gen)
        if op == "route":
            s["bias"] = randn(E, std=0.1) if case["bias"] else None
            s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["w"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
        else:
            full = dict(case, groups=1, keep=1, top2=False)
            s["ids"], s["w"] = _plain_route(full, s["logits"], None)
            s["d_w"] = randn(T, k)
            s["d_logits"] = torch.empty_like(s["logits"])
    elif op == "scale_back":
        T, d, k = case["tokens"], case["hidden"], case["top_k"]
        E = 32
        ids = torch.rand(T, E, generator=gen, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
        s["w"] = torch.softmax(randn(T, k), 1)
        s["recv"] = randn(T * k, d, dtype=torch.bfloat16)
        s["d_out"] = randn(T, d, dtype=torch.bfloat16)
        s["d_recv"] = torch.empty_like(s["recv"])
        s["d_w"] = torch.empty_like(s["w"])
        # receive rows are ordered by (expert, token)
        s["pos"] = ids.reshape(-1).long().argsort(stable=True).argsort().view(T, k)
        s["ids"] = ids
        if own:
            # the plan that the forward pass of the same step has made
            import moe_expert_tile_amd as m
            s["shape"] = m.Shape(1, 0, E, k, d, 128, 32, [T], T * k)
            s["plan"] = torch.zeros(m.moe_query_sizes(s["shape"])["plan_bytes"] // 4, dtype=torch.int32, device="cuda")
            m.moe_plan(s["shape"], ids, s["recv"], s["plan"], None)
    else:
        M, N, K = case["rows"], case["cols"], case["depth"]
        t, o = _TYPES[case["dtype"]], _TYPES[case["out"]]
        NZ = 2 * N if case["act"] == "swiglu" else N
        s["x"] = randn(M, K, dtype=t)
        s["weight"] = randn(NZ, K, std=K ** -0.5, dtype=t)
        if op == "linear":
            s["bias"] = randn(NZ, std=0.5, dtype=t) if case["bias"] else None
            s["residual"] = randn(M, N, dtype=o) if case["residual"] else None
            s["pre"] = torch.empty(M, NZ, dtype=t, device="cuda") if case["pre"] else None
            s["out"] = torch.empty(M, N, dtype=o, device="cuda")
        else:
            s["pre"] = randn(M, NZ, dtype=t) if case["act"] != "none" else None
            s["d_out"] = randn(M, N, dtype=o)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty_like(s["weight"])
            s["db"] = torch.empty(NZ, dtype=t, device="cuda") if case["bias"] else None
    return s


# --- plain forms -------------------------------------------------------------

def _plain_scores(case, z):
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True).clamp_min(1e-300)


def _plain_route(case, logits, bias):
    # the choice between near scores hangs on their last bits: 64
    z = logits.double()
    T, E = z.shape
    k = case["top_k"]
    s = _plain_scores(case, z)
    c = s if bias is None else s + bias.double()
    c = torch.where(torch.isneginf(z), z, c)
    G = case["groups"]
    if G > 1:
        best = c.view(T, G, E // G).sort(dim=2, descending=True).values
        group = best[:, :, 0] + best[:, :, 1] if case["top2"] else best[:, :, 0]
        chosen = group.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=z.device)
        kept[torch.arange(T, device=z.device)[:, None], chosen] = True
        c = torch.where(kept[:, :, None].expand(T, G, E // G).reshape(T, E), c, -math.inf)
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.where(torch.isneginf(c.gather(1, ids)), 0.0, s.gather(1, ids))
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.to(torch.int32), (w * case["scale"]).float()


def _plain_route_back(case, logits, ids, w, d_w):
    z, ids = logits.float(), ids.long()
    live = (w != 0).float()
    g = d_w * live
    s = _plain_scores(case, z.double()).float()
    sel = s.gather(1, ids) * live
    scale = case["scale"]
    ds = scale * g
    if case["renorm"]:
        total = sel.sum(1, keepdim=True)
        ds = torch.where(total > 0, scale * (g - (g * sel / total).sum(1, keepdim=True)) / total, 0.0) * live
    if case["score"] == "sigmoid":
        flow = torch.where(live > 0, ds * sel * (1 / (1 + torch.exp(z.gather(1, ids)))), 0.0)
        dz = torch.zeros_like(z).scatter_add(1, ids, flow)
    else:
        dz = torch.zeros_like(z).scatter_add(1, ids, ds * sel) - s * (ds * sel).sum(1, keepdim=True)
    return dz.to(logits.dtype)


def _plain_act(act, z):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _plain_slope(act, z):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi)
        t = torch.tanh(u * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * u * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s):
    case = s["case"]
    z = s["x"].float() @ s["weight"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if case["act"] == "swiglu":
        N = case["cols"]
        out = _plain_act("silu", z[:, :N]) * z[:, N:]
    else:
        out = _plain_act(case["act"], z)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    got = {"out": out.to(s["out"].dtype)}
    if s["pre"] is not None:
        got["pre"] = z.to(s["pre"].dtype)
    return got


def _plain_linear_back(s):
    case = s["case"]
    g = s["d_out"].float()
    if case["act"] == "swiglu":
        gate, up = s["pre"].float().chunk(2, 1)
        dz = torch.cat([g * up * _plain_slope("silu", gate), g * _plain_act("silu", gate)], 1)
    elif case["act"] == "none":
        dz = g
    else:
        dz = g * _plain_slope(case["act"], s["pre"].float())
    got = {"dx": (dz @ s["weight"].float()).to(s["x"].dtype), "dw": (dz.t() @ s["x"].float()).to(s["weight"].dtype)}
    if s["db"] is not None:
        got["db"] = dz.sum(0).to(s["db"].dtype)
    return got


def _plain_scale_back(s):
    T, k = s["w"].shape
    g, pos = s["d_out"].float(), s["pos"]
    d_w = (s["recv"].float()[pos] * g[:, None, :]).sum(2)
    d_recv = torch.empty_like(s["recv"])
    d_recv[pos.reshape(-1)] = (s["w"][:, :, None] * g[:, None, :]).to(torch.bfloat16).view(T * k, -1)
    return {"d_recv": d_recv, "d_w": d_w}


# --- one pass ----------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s)
    if op == "route":
        ids, w = _plain_route(case, s["logits"], s["bias"])
        return {"ids": ids, "w": w}
    if op == "route_back":
        return {"d_logits": _plain_route_back(case, s["logits"], s["ids"], s["w"], s["d_w"])}
    if op == "scale_back":
        return _plain_scale_back(s)
    return _plain_linear(s) if op == "linear" else _plain_linear_back(s)


def _own(s):
    import moe_expert_tile_amd as m
    case = s["case"]
    op = case["op"]
    if op in ("route", "route_back"):
        score = m.SCORE_SIGMOID if case["score"] == "sigmoid" else m.SCORE_SOFTMAX
        if op == "route":
            m.moe_route(s["logits"], s["ids"], s["w"], bias=s["bias"], score=score, renorm=case["renorm"],
                        n_group=case["groups"], topk_group=case["keep"],
                        group_score=m.GROUP_TOP2 if case["top2"] else m.GROUP_MAX, scale=case["scale"])
            return {"ids": s["ids"], "w": s["w"]}
        m.moe_route_backward(s["logits"], s["ids"], s["w"], s["d_w"], s["d_logits"], score=score,
                             renorm=case["renorm"], scale=case["scale"])
        return {"d_logits": s["d_logits"]}
    if op == "scale_back":
        m.moe_scale_backward(s["shape"], s["plan"], s["recv"], s["w"], s["d_out"], s["d_recv"], s["d_w"])
        return {"d_recv": s["d_recv"], "d_w": s["d_w"]}
    act = getattr(m, "ACT_" + case["act"].upper())
    if op == "linear":
        m.moe_linear(s["x"], s["weight"], s["out"], bias=s["bias"], residual=s["residual"], pre=s["pre"], act=act)
        return {"out": s["out"]} if s["pre"] is None else {"out": s["out"], "pre": s["pre"]}
    m.moe_linear_backward(s["x"], s["weight"], s["d_out"], dx=s["dx"], dw=s["dw"], dbias=s["db"], pre=s["pre"], act=act)
    got = {"dx": s["dx"], "dw": s["dw"]}
    if s["db"] is not None:
        got["db"] = s["db"]
    return got


# --- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    if op in ("route", "route_back"):
        T, E, k, b = case["tokens"], case["experts"], case["top_k"], _SIZE[case["dtype"]]
        if op == "route":
            # the logits in, ids and weights out; a score and a comparison each
            return {"bytes": T * E * b + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
        reads = T * E * b if case["score"] == "softmax" and not case["renorm"] else T * k * b
        return {"bytes": reads + 12 * T * k + T * E * b, "flops": 8 * T * k}
    if op == "scale_back":
        T, d, k = case["tokens"], case["hidden"], case["top_k"]
        return {"bytes": 2 * T * d + 4 * T * k * d + 12 * T * k, "flops": 3 * T * k * d}
    M, N, K = case["rows"], case["cols"], case["depth"]
    NZ = 2 * N if case["act"] == "swiglu" else N
    b, o = _SIZE[case["dtype"]], _SIZE[case["out"]]
    if op == "linear":
        extra = (NZ * b if case["bias"] else 0) + (M * N * o if case["residual"] else 0) + (M * NZ * b if case["pre"] else 0)
        return {"bytes": (M * K + NZ * K) * b + M * N * o + extra, "flops": 2 * M * NZ * K}
    extra = (M * NZ * b if case["act"] != "none" else 0) + (NZ * b if case["bias"] else 0)
    return {"bytes": 2 * (M * K + NZ * K) * b + M * N * o + extra, "flops": 4 * M * NZ * K}


# --- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, s["logits"].double().cpu().numpy(),
                            None if s["bias"] is None else s["bias"].double().cpu().numpy())
    if op == "route_back":
        return _exact_route_back(case, s["logits"].double().cpu().numpy(), s["ids"].cpu().numpy(),
                                 s["w"].cpu().numpy(), s["d_w"].double().cpu().numpy())
    if op == "scale_back":
        d_w = torch.empty(s["w"].shape, dtype=torch.float64, device="cuda")
        d_recv = torch.empty(s["recv"].shape, dtype=torch.float64, device="cuda")
        g = s["d_out"].double()
        for j in range(case["top_k"]):
            rows = s["pos"][:, j]
            d_w[:, j] = torch.einsum("td,td->t", s["recv"][rows].double(), g)
            d_recv[rows] = s["w"][:, j].double().unsqueeze(1) * g
        return {"d_recv": d_recv, "d_w": d_w}
    x, weight = s["x"].double(), s["weight"].double()
    N, act = case["cols"], case["act"]
    if op == "linear":
        z = torch.mm(x, weight.t().contiguous())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act("silu", z[:, :N])[0] * z[:, N:] if act == "swiglu" else _exact_act(act, z)[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"out": y, "pre": z} if case["pre"] else {"out": y}
    g = s["d_out"].double()
    if act == "swiglu":
        p = s["pre"].double()
        value, slope = _exact_act("silu", p[:, :N])
        dz = torch.cat((g * p[:, N:] * slope, g * value), 1)
    else:
        dz = g if act == "none" else g * _exact_act(act, s["pre"].double())[1]
    got = {"dx": torch.mm(dz, weight), "dw": torch.mm(dz.t().contiguous(), x)}
    if case["bias"]:
        got["db"] = dz.sum(0)
    return got


def _exact_route(case, z, bias):
    T, E = z.shape
    if case["score"] == "softmax":
        lse = np.logaddexp.reduce(z, axis=1, keepdims=True)
        with np.errstate(invalid="ignore"):
            p = np.where(np.isneginf(z), 0.0, np.exp(z - lse))
    else:
        p = np.exp(-np.logaddexp(0.0, -z))
    rank = p.copy() if bias is None else p + bias[None, :]
    rank[z == -np.inf] = -np.inf
    G = case["groups"]
    if G > 1:
        parts = np.sort(rank.reshape(T, G, -1), axis=2)
        score = parts[:, :, -1] + (parts[:, :, -2] if case["top2"] else 0.0)
        place = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1, kind="stable")
        rank = np.where(np.repeat(place >= case["keep"], E // G, axis=1), -np.inf, rank)
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :case["top_k"]]
    w = np.take_along_axis(p, ids, 1)
    w[np.isneginf(np.take_along_axis(rank, ids, 1))] = 0.0
    if case["renorm"]:
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    return {"ids": ids.astype(np.int32), "w": w * case["scale"]}


def _exact_route_back(case, z, ids, w, d_w):
    # the Jacobian of the weights, applied to their gradient: w = scale p / S (or scale p)
    T, E = z.shape
    rows = np.arange(T)[:, None]
    held = w != 0
    if case["score"] == "softmax":
        lse = np.logaddexp.reduce(z, axis=1, keepdims=True)
        with np.errstate(invalid="ignore"):
            p = np.where(np.isneginf(z), 0.0, np.exp(z - lse))
    else:
        p = np.exp(-np.logaddexp(0.0, -z))
    ps = np.where(held, p[rows, ids], 0.0)
    g = np.where(held, d_w, 0.0) * case["scale"]
    if case["renorm"]:
        total = ps.sum(1, keepdims=True)
        total = np.where(total > 0, total, 1.0)
        g = np.where(held, (g - (g * ps).sum(1, keepdims=True) / total) / total, 0.0)
    dp = np.zeros((T, E))
    np.add.at(dp, (rows, ids), g)
    if case["score"] == "softmax":
        return {"d_logits": p * (dp - (dp * p).sum(1, keepdims=True))}
    return {"d_logits": dp * p * np.exp(-np.logaddexp(0.0, z))}


def _exact_act(act, z):
    """(value, slope) of an activation at z."""
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2u
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z.pow(3)))
        return z * p, p + z * p * (1 - p) * c * (1 + 0.134145 * z.square())
    return z, torch.ones_like(z)
