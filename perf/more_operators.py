"""The measured calls of the sorted experts' rows and their 4-bit products:
sorting a batch's (token, slot) pairs by expert (moe_sort), its tokens to the
experts' rows and back with their gradients (moe_permute, moe_unpermute),
microscaled 4-bit rows (moe_mx_quantize, moe_mx_dequantize) and the product
with such weights, expert by expert (moe_mx_linear).

Each case is one pass as a user's program makes it.  With ``own`` false the
operators are computed in plain torch operations in 32 bits; with ``own`` true
by the library's entry points.  ``exact`` computes the same from the
definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_BLOCK = 32   # elements that share a scale


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step: 64 tokens over 128 experts; latency of a short call
        {"name": "sort_decode", "op": "sort", "tokens": 64, "total": 128, "first": 0, "experts": 128, "top_k": 8},
        # a long prefill over all of a layer's experts
        {"name": "sort_prefill", "op": "sort", "tokens": 32768, "total": 256, "first": 0, "experts": 256, "top_k": 8},
        # a ragged batch of odd rows to the experts of one rank; a fifth of the slots belong to others
        {"name": "permute_ragged", "op": "permute", "tokens": 777, "cols": 1001, "top_k": 6, "dtype": "f16",
         "dropped": 0.2},
        # the gradient of a training batch's tokens from its experts' rows
        {"name": "permute_back_train", "op": "permute_back", "tokens": 8192, "cols": 4096, "top_k": 8, "dtype": "bf16",
         "dropped": 0.0},
        # a decode step's weighted sum of its experts' rows
        {"name": "unpermute_decode", "op": "unpermute", "tokens": 64, "cols": 2048, "top_k": 8, "dtype": "bf16",
         "dropped": 0.0, "weighted": True},
        # the gradients of that sum for a training batch of wide rows
        {"name": "unpermute_back_train", "op": "unpermute_back", "tokens": 4097, "cols": 7168, "top_k": 8,
         "dtype": "bf16", "dropped": 0.0, "weighted": True},
        # a decode step's activations to 4 bits and back
        {"name": "mx_round_decode", "op": "mx_round", "rows": 64, "depth": 2048, "dtype": "bf16"},
        # ... and a prefill's
        {"name": "mx_round_prefill", "op": "mx_round", "rows": 16384, "depth": 7168, "dtype": "bf16"},
        # one token through its 8 of 64 experts' gated up projections: the weights' bytes and the launch
        {"name": "mx_token", "op": "mx_linear", "rows": 8, "spare": 0, "experts": 64, "hit": 8, "cols": 2048,
         "depth": 7168, "dtype": "bf16", "out": "bf16", "act": "swiglu", "bias": False},
        # a decode step of 64 tokens, 8 slots each, over 128 small experts
        {"name": "mx_decode", "op": "mx_linear", "rows": 512, "spare": 0, "experts": 128, "hit": 128, "cols": 768,
         "depth": 2048, "dtype": "bf16", "out": "bf16", "act": "swiglu", "bias": False},
        # a prefill's rows in 16 bits over 16 experts: 4-bit weights alone
        {"name": "mx_prefill", "op": "mx_linear", "rows": 16384, "spare": 0, "experts": 16, "hit": 16, "cols": 1536,
         "depth": 4096, "dtype": "bf16", "out": "bf16", "act": "swiglu", "bias": False},
        # a long prefill with rows and weights in 4 bits over 32 experts, some rows of the buffer unused
        {"name": "mx_prefill_both", "op": "mx_linear", "rows": 46451, "spare": 85, "experts": 32, "hit": 32,
         "cols": 2048, "depth": 7168, "dtype": "mx", "out": "bf16", "act": "swiglu", "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "permute", "permute_back", "unpermute", "unpermute_back", "mx_round", "mx_linear",
                     "mx_linear", "mx_linear"])
    if op == "sort":
        tokens, total = _log(rng, 4, 32768), _log(rng, 8, 512)
        # all experts, or one rank's share of them
        experts = rng.choice([total, total, total // rng.choice([2, 4, 8])]) if tokens > 64 else total
        return {"op": op, "tokens": tokens, "total": total, "first": rng.randint(0, total - experts),
                "experts": experts, "top_k": rng.randint(1, min(8, total))}
    if op in ("permute", "permute_back", "unpermute", "unpermute_back"):
        cols, top_k, dtype = _log(rng, 8, 7168), rng.randint(1, 8), rng.choice(["bf16", "bf16", "f16", "f32"])
        most = 4097 * 7168 * 8 * 2 // (_SIZE[dtype] * cols * top_k)
        tokens = _log(rng, 1, min(16384, most))
        c = {"op": op, "tokens": tokens, "cols": cols, "top_k": top_k, "dtype": dtype,
             "dropped": rng.choice([0.0, 0.0, 0.2, 0.7]) if tokens > 32 else 0.0}
        if op.startswith("un"):
            c["weighted"] = rng.random() < 0.8
        return c
    if op == "mx_round":
        return {"op": op, "rows": _log(rng, 1, 8192), "depth": _BLOCK * _log(rng, 1, 224),
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    act = rng.choice(["none", "silu", "swiglu", "swiglu"])
    cols, depth = _log(rng, 8, 4096), _BLOCK * _log(rng, 1, 224)
    if act == "swiglu":
        cols = (cols + 1) // 2
    most = 32 * 4096 * 7168 // ((2 if act == "swiglu" else 1) * cols * depth)
    experts = _log(rng, 1, max(1, min(128, most)))
    rows = _log(rng, 1, 16384)
    dtype = rng.choice(["bf16", "f16", "mx", "mx"])
    return {"op": op, "rows": rows, "spare": rng.choice([0, 0, rng.randint(1, 64)]), "experts": experts,
            "hit": min(rows, rng.choice([experts, max(1, experts // 2)])), "cols": cols, "depth": depth,
            "dtype": dtype, "out": rng.choice(["f32", "f16" if dtype == "f16" else "bf16"]), "act": act,
            "bias": rng.random() < 0.4}


# --- inputs ------------------------------------------------------------------

def _times(x, e):
    """x times 2^e, exactly (a library's power of two need not be)."""
    return x * ((e.long() + 1023) << 52).view(torch.float64).float()


def _pack(x):
    """Rows in microscaled 4 bits: (codes, two a byte, the even element's in the
    low half; a byte 127 + log2 of the scale for each 32 elements)."""
    v = x.view(*x.shape[:-1], -1, _BLOCK)
    top = v.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    y = _times(v, -e.unsqueeze(-1))
    a = y.abs()
    code = (a > 0.25).to(torch.uint8)
    for bar, over in ((0.75, torch.ge), (1.25, torch.gt), (1.75, torch.ge), (2.5, torch.gt), (3.5, torch.ge), (5.0, torch.gt)):
        code += over(a, bar)
    code += 8 * (y < 0)
    code = code.view(*x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op == "sort":
        T, E, k, total = case["tokens"], case["experts"], case["top_k"], case["total"]
        # distinct experts a token, some of them favoured
        score = torch.rand(T, total, generator=gen, device="cuda").log().neg_().log_().neg_()
        score += randn(total)
        s["ids"] = score.topk(k, dim=1).indices.to(torch.int32).contiguous()
        s["pos"] = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        s["src"] = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    elif op in ("permute", "permute_back", "unpermute", "unpermute_back"):
        T, d, k, t = case["tokens"], case["cols"], case["top_k"], _TYPES[case["dtype"]]
        # places of the slots: a sort by expert, the dropped ones nowhere
        key = torch.randint(0, 64, (T * k,), generator=gen, device="cuda")
        key[torch.rand(T * k, generator=gen, device="cuda") < case["dropped"]] = 64
        place = key.argsort(stable=True).argsort()
        s["pos"] = torch.where(key < 64, place, -1).to(torch.int32).view(T, k)
        held = (key < 64).sum()
        live = (torch.arange(T * k, device="cuda") < held).unsqueeze(1)
        rows = lambda: torch.where(live, randn(T * k, d), 0).to(t)  # noqa: E731
        s["w"] = torch.softmax(randn(T, k), 1) if case.get("weighted") else None
        if op == "permute":
            s["x"], s["rows"] = randn(T, d, dtype=t), torch.zeros(T * k, d, dtype=t, device="cuda")
        elif op == "permute_back":
            s["d_rows"], s["dx"] = rows(), torch.empty(T, d, dtype=t, device="cuda")
        elif op == "unpermute":
            s["rows"], s["out"] = rows(), torch.empty(T, d, dtype=t, device="cuda")
        else:
            s["rows"], s["d_out"] = rows(), randn(T, d, dtype=t)
            s["d_rows"] = torch.zeros(T * k, d, dtype=t, device="cuda")
            s["d_w"] = torch.empty(T, k, device="cuda") if s["w"] is not None else None
    elif op == "mx_round":
        M, K, t = case["rows"], case["depth"], _TYPES[case["dtype"]]
        # activations: a few loud channels, tokens of differing size
        x = randn(M, K) * torch.exp(0.5 * randn(M, 1))
        x *= 1 + 15 * (torch.rand(K, generator=gen, device="cuda") < 0.01)
        s["x"] = x.to(t)
        s["q"] = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty(M, K // _BLOCK, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty(M, K, dtype=t, device="cuda")
    else:
        M, N, K, E = case["rows"], case["cols"], case["depth"], case["experts"]
        n = 2 * N if case["act"] == "swiglu" else N
        x = randn(M + case["spare"], K)
        if case["dtype"] == "mx":
            s["x"], s["x_scale"] = _pack(x)
        else:
            s["x"], s["x_scale"] = x.to(_TYPES[case["dtype"]]), None
        s["w"] = torch.empty(E, n, K // 2, dtype=torch.uint8, device="cuda")
        s["w_scale"] = torch.empty(E, n, K // _BLOCK, dtype=torch.uint8, device="cuda")
        for e in range(E):
            s["w"][e], s["w_scale"][e] = _pack(randn(n, K, std=K ** -0.5))
        s["bias"] = randn(E, n, std=0.5, dtype=_TYPES[case["out"]]) if case["bias"] else None
        # rows an expert: one at least for those that are hit, the rest by uneven chances
        hit = torch.randperm(E, generator=gen, device="cuda")[:case["hit"]]
        more = torch.multinomial(torch.exp(0.7 * randn(case["hit"])), M - case["hit"], replacement=True, generator=gen) \
            if M > case["hit"] else hit[:0]
        count = torch.zeros(E, dtype=torch.int64, device="cuda")
        count[hit] = 1 + torch.bincount(more, minlength=case["hit"])
        s["offsets"] = torch.nn.functional.pad(count.cumsum(0), (1, 0)).to(torch.int32)
        s["bounds"] = s["offsets"].tolist()
        s["out"] = torch.zeros(M + case["spare"], N, dtype=_TYPES[case["out"]], device="cuda")
    return s


# --- plain forms -------------------------------------------------------------

def _plain_sort(s):
    case, ids = s["case"], s["ids"].reshape(-1).long()
    E, P = case["experts"], ids.numel()
    local = ids - case["first"]
    key = torch.where((local >= 0) & (local < E), local, E)
    order = key.sort(stable=True).indices
    offsets = torch.nn.functional.pad(torch.bincount(key, minlength=E + 1).cumsum(0)[:E], (1, 0))
    place = torch.empty_like(order)
    place[order] = torch.arange(P, device=ids.device)
    pos = torch.where(key < E, place, -1).view(s["ids"].shape)
    src = torch.where(torch.arange(P, device=ids.device) < offsets[E], order, -1)
    return {"pos": pos.to(torch.int32), "src": src.to(torch.int32), "offsets": offsets.to(torch.int32)}


def _plain_rows(s):
    case, pos = s["case"], s["pos"].long()
    op, (T, k) = case["op"], s["pos"].shape
    P, d = T * k, case["cols"]
    to = torch.where(pos < 0, P, pos)              # one row more takes and gives what is dropped
    if op == "permute":
        rows = torch.zeros(P + 1, d, dtype=s["x"].dtype, device=pos.device)
        rows[to.reshape(-1)] = s["x"].unsqueeze(1).expand(T, k, d).reshape(P, d)
        return {"rows": rows[:P]}
    given = s["d_rows"] if op == "permute_back" else s["rows"]
    held = torch.nn.functional.pad(given, (0, 0, 0, 1))[to].float()
    if op == "permute_back":
        return {"dx": held.sum(1).to(given.dtype)}
    w = s["w"]
    if op == "unpermute":
        return {"out": (held if w is None else w.unsqueeze(2) * held).sum(1).to(given.dtype)}
    g = s["d_out"].float().unsqueeze(1)
    d_rows = torch.zeros(P + 1, d, dtype=given.dtype, device=pos.device)
    d_rows[to.reshape(-1)] = (g.expand(T, k, d) if w is None else w.unsqueeze(2) * g).to(given.dtype).reshape(P, d)
    if w is None:
        return {"d_rows": d_rows[:P]}
    return {"d_rows": d_rows[:P], "d_w": (held * g).sum(2)}


def _plain_round(x):
    """The nearest values with one bit behind the leading one, of a block's scale."""
    v = x.float().view(x.shape[0], -1, _BLOCK)
    e = (torch.frexp(v.abs().amax(-1, keepdim=True)).exponent - 3).clamp(-127, 127)
    y = _times(v, -e)
    step = (torch.frexp(y).exponent - 2).clamp_min(-1)
    r = _times(torch.round(_times(y, -step)), step).clamp(-6, 6)
    return _times(r, e).view(x.shape).to(x.dtype)


def _values(q, scale):
    """What packed rows stand for, in 32 bits."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    code = torch.stack((q & 15, q >> 4), -1).view(*q.shape[:-1], -1, _BLOCK).int()
    return _times(table[code], scale.unsqueeze(-1).long() - 127).flatten(-2)


def _plain_linear(s):
    case, N = s["case"], s["case"]["cols"]
    x = s["x"].float() if s["x_scale"] is None else _values(s["x"], s["x_scale"])
    out = torch.zeros_like(s["out"])
    # expert by expert, one product each
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if lo == hi:
            continue
        z = x[lo:hi] @ _values(s["w"][e], s["w_scale"][e]).t()
        if s["bias"] is not None:
            z += s["bias"][e].float()
        if case["act"] == "swiglu":
            z = z[:, :N] / (1 + torch.exp(-z[:, :N])) * z[:, N:]
        elif case["act"] == "silu":
            z = z / (1 + torch.exp(-z))
        out[lo:hi] = z
    return {"out": out}


# --- one pass ----------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "sort":
        return _plain_sort(s)
    if op == "mx_round":
        return {"values": _plain_round(s["x"])}
    return _plain_linear(s) if op == "mx_linear" else _plain_rows(s)


def _own(s):
    import moe_expert_tile_amd as m
    case = s["case"]
    op = case["op"]
    if op == "sort":
        m.moe_sort(s["ids"], s["pos"], s["offsets"], src=s["src"], first=case["first"])
        return {"pos": s["pos"], "src": s["src"], "offsets": s["offsets"]}
    if op == "permute":
        m.moe_permute(s["x"], s["pos"], s["rows"])
        return {"rows": s["rows"]}
    if op == "permute_back":
        m.moe_permute_backward(s["d_rows"], s["pos"], s["dx"])
        return {"dx": s["dx"]}
    if op == "unpermute":
        m.moe_unpermute(s["rows"], s["pos"], s["out"], topk_w=s["w"])
        return {"out": s["out"]}
    if op == "unpermute_back":
        m.moe_unpermute_backward(s["pos"], s["d_out"], rows=s["rows"], topk_w=s["w"], d_rows=s["d_rows"], d_topk_w=s["d_w"])
        return {"d_rows": s["d_rows"]} if s["d_w"] is None else {"d_rows": s["d_rows"], "d_w": s["d_w"]}
    if op == "mx_round":
        m.moe_mx_quantize(s["x"], s["q"], s["scale"])
        m.moe_mx_dequantize(s["q"], s["scale"], s["values"])
        return {"values": s["values"]}
    m.moe_mx_linear(s["x"], s["w"], s["w_scale"], s["out"], offsets=s["offsets"], x_scale=s["x_scale"], bias=s["bias"],
                    act=getattr(m, "ACT_" + case["act"].upper()))
    return {"out": s["out"]}


# --- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    if op == "sort":
        P = case["tokens"] * case["top_k"]
        return {"bytes": 12 * P + 4 * (case["experts"] + 1), "flops": P}
    if op in ("permute", "permute_back", "unpermute", "unpermute_back"):
        T, k, d, b = case["tokens"], case["top_k"], case["cols"], _SIZE[case["dtype"]]
        R = round(T * k * (1 - case["dropped"]))
        w = 4 * T * k if case.get("weighted") else 0
        if op == "unpermute_back":
            # the rows are read for the weights' gradient alone
            return {"bytes": b * d * (T + R * (2 if w else 1)) + 4 * T * k + 2 * w, "flops": 3 * R * d if w else R * d}
        return {"bytes": b * d * (T + R) + 4 * T * k + w, "flops": 0 if op == "permute" else 2 * R * d}
    if op == "mx_round":
        n, b = case["rows"] * case["depth"], _SIZE[case["dtype"]]
        # the values in and out, the packed rows written and read
        return {"bytes": 2 * b * n + 2 * (n // 2 + n // _BLOCK), "flops": 4 * n}
    M, N, K = case["rows"], case["cols"], case["depth"]
    n = 2 * N if case["act"] == "swiglu" else N
    packed = lambda r: r * (K // 2 + K // _BLOCK)  # noqa: E731
    x = packed(M) if case["dtype"] == "mx" else 2 * M * K
    o = _SIZE[case["out"]]
    return {"bytes": x + case["hit"] * (packed(n) + (n * o if case["bias"] else 0)) + M * N * o + 4 * (case["experts"] + 1),
            "flops": 2 * M * n * K}


# --- the definitions in 64 bits ----------------------------------------------

def _power(e):
    """2^e of whole numbers from -300 to 300."""
    table = torch.tensor([math.ldexp(1.0, i) for i in range(-300, 301)], dtype=torch.float64, device=e.device)
    return table[e.long() + 300]


def _exact_values(q, scale):
    """Sign, two exponent bits and one fraction bit, times 2^(scale - 127)."""
    code = torch.stack((q % 16, q // 16), -1).flatten(-2).long()
    power, half = code // 2 % 4, code % 2
    size = torch.where(power > 0, (1 + 0.5 * half.double()) * _power(power - 1), 0.5 * half.double())
    size = torch.where(code > 7, -size, size)
    return size * _power(scale.long() - 127).repeat_interleave(_BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        # each slot's place: slots of lower experts, and earlier ones of its own
        ids = s["ids"].view(-1).cpu().long().numpy() - case["first"]
        E, at = case["experts"], 0
        pos, src, offsets = torch.full((ids.size,), -1), torch.full((ids.size,), -1), torch.zeros(E + 1)
        for e in range(E):
            slots = torch.from_numpy((ids == e).nonzero()[0])
            pos[slots] = torch.arange(at, at + len(slots))
            src[at:at + len(slots)] = slots
            at += len(slots)
            offsets[e + 1] = at
        return {"pos": pos.view(s["pos"].shape).int(), "src": src.int(), "offsets": offsets.int()}
    if op == "mx_round":
        x = s["x"].double()
        blocks = x.view(x.shape[0], -1, _BLOCK)
        top = blocks.abs().amax(-1, keepdim=True)
        power = torch.floor(torch.log2(top.clamp_min(2.0 ** -200)))
        power += (_power(power + 1) <= top).double() - (_power(power) > top).double()     # log2 rounds near powers of two
        unit = _power((power - 2).clamp(-127, 127))
        a, r = blocks.abs() / unit, torch.zeros_like(blocks)
        for below, value, even in ((0.25, 0.5, 0), (0.75, 1, 1), (1.25, 1.5, 0), (1.75, 2, 1), (2.5, 3, 0), (3.5, 4, 1), (5, 6, 0)):
            r = torch.where((a >= below) if even else (a > below), float(value), r)
        return {"values": (torch.sign(blocks) * r * unit).view(x.shape)}
    if op == "mx_linear":
        x = s["x"].double() if s["x_scale"] is None else _exact_values(s["x"], s["x_scale"])
        N, out = case["cols"], torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            lo, hi = s["bounds"][e], s["bounds"][e + 1]
            if hi == lo:
                continue
            z = torch.mm(x[lo:hi], _exact_values(s["w"][e], s["w_scale"][e]).t().contiguous())
            if case["bias"]:
                z += s["bias"][e].double()
            if case["act"] == "none":
                out[lo:hi] = z
            else:
                gate = z[:, :N]
                out[lo:hi] = gate * torch.sigmoid(gate) * (z[:, N:] if case["act"] == "swiglu" else 1)
        return {"out": out}
    T, k = s["pos"].shape
    shape = (T * k, case["cols"])
    pos, w = s["pos"].long(), s["w"]
    if op == "permute":
        rows = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            there = pos[:, j] >= 0
            rows[pos[there, j]] = s["x"][there].double()
        return {"rows": rows}
    if op == "unpermute_back":
        d_rows, d_w = torch.zeros(shape, dtype=torch.float64, device="cuda"), torch.zeros(T, k, dtype=torch.float64, device="cuda")
        g = s["d_out"].double()
        for j in range(k):
            there = pos[:, j] >= 0
            at = pos[there, j]
            d_rows[at] = g[there] if w is None else w[there, j].double().unsqueeze(1) * g[there]
            d_w[there, j] = torch.einsum("td,td->t", s["rows"][at].double(), g[there])
        return {"d_rows": d_rows} if w is None else {"d_rows": d_rows, "d_w": d_w}
    given = s["rows"] if op == "unpermute" else s["d_rows"]
    out = torch.zeros(T, case["cols"], dtype=torch.float64, device="cuda")
    for j in range(k):
        there = pos[:, j] >= 0
        part = given[pos[there, j]].double()
        out[there] += part if w is None else w[there, j].double().unsqueeze(1) * part
    return {"out": out} if op == "unpermute" else {"dx": out}
