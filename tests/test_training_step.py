"""A training step around the sorted rows: sort, rows, each expert's dense
products, the weighted sum, and back.  Every entry of the gradients of the
tokens, the experts' weights and the logits is held against its formula in
float64; the formulas against differences; and the bounds against planted
mistakes, which they refuse.

The bounds follow the chain.  With u = 2^-24, h = 2^-11 (half a step of fp16) and
t = 2^-25 (half a step of its smallest values), a value v known up to e and
rounded to fp16 is known up to (1 + h) e + h |v| + t; a product of a, b known up to ea, eb
up to (|a| + ea) (|b| + eb) - |a| |b|; an fp32 sum of n products adds (n + 8) u
of the sum of their magnitudes.  The gate's slope is at most 1.13 and its
slope's slope at most 1/2.  The routing's weights are good to 2^-18, its
gradient to 2^-17 of the token's largest d_w; the dense products' gradients
scale dz so that a rounding is off by 2^-39 of the largest one, if that is more than h
of its value."""
import numpy as np
import pytest

from oracle import linear as OL
from oracle import route as OR
from oracle import rows as OS
from oracle import step as ST

H, T16, U = 2.0 ** -11, 2.0 ** -25, 2.0 ** -24


def inputs(kind, T=48, total=8, E=5, k=2, d=32, f=24, seed=0):
    """Token, weight and gradient values in fp16.  "signed": sums cancel; "positive": they do not, and experts differ."""
    rng = np.random.default_rng(seed)
    f16 = lambda a: a.astype(np.float16).astype(np.float64)  # noqa: E731
    x, up, down, g = rng.standard_normal((T, d)), rng.standard_normal((E, 2 * f, d)), rng.standard_normal((E, d, f)), rng.standard_normal((T, d))
    if kind == "positive":
        x, up, down, g = abs(x), abs(up) * (0.3 + np.arange(E)[:, None, None]) / 3, abs(down), abs(g)
    logits = rng.standard_normal((T, total)).astype(np.float32).astype(np.float64)
    return dict(x=f16(x), up=f16(0.2 * up), down=f16(0.2 * down), g=f16(g), logits=logits, ids=OR.route(logits, k, renorm=True)[0], first=2)


class _Known:
    """A value and the most it can be off by."""

    def __init__(self, v, e):
        self.v, self.e = v, e

    @property
    def top(self):
        return np.abs(self.v) + self.e

    def half(self, least=T16):
        """Rounded to fp16."""
        return _Known(self.v, (1 + H) * self.e + H * np.abs(self.v) + least)


def _product(a, b, n):
    """a b^T summed in fp32 over n entries."""
    v, size, top = a.v @ b.v.T, np.abs(a.v) @ np.abs(b.v).T, a.top @ b.top.T
    return _Known(v, top - size + (n + 8) * U * top)


def _turned(a):
    return _Known(a.v.T, a.e.T)


def bounds(a):
    """{name: (gradient, the most an entry can be off by)}, with the gradients taken step by step."""
    x, up, down, g, ids, first = (a[n] for n in ("x", "up", "down", "g", "ids", "first"))
    E, f, d = len(up), up.shape[1] // 2, x.shape[1]
    k = ids.shape[1]
    w = OR.weights_of(a["logits"], ids, np.ones(ids.shape, bool), "softmax", True)
    exact = lambda v: _Known(v, np.zeros_like(v))  # noqa: E731
    out = {n: (np.zeros_like(v), np.zeros_like(v)) for n, v in (("dx", x), ("d_up", up), ("d_down", down))}
    d_w = _Known(np.zeros(ids.shape), np.zeros(ids.shape))
    d_rows = []                       # (token, gradient) of the rows
    for e in range(E):
        at = np.argwhere(ids == e + first)
        if not len(at):
            continue
        t, j = at.T
        xr, gr, wr = exact(x[t]), g[t], w[t, j][:, None]
        z = _product(xr, exact(up[e]), d)
        zg, zu = (_Known(z.v[:, s], z.e[:, s]) for s in (slice(None, f), slice(f, None)))
        s = OL.activation("silu", zg.v)
        h = _Known(s * zu.v, (np.abs(s) + 1.13 * zg.e) * zu.top - np.abs(s * zu.v) + (16 + 64 * zg.top) * U * (np.abs(s) + 1.13 * zg.e) * zu.top).half()
        pre = _Known(z.v, z.e).half()
        y = _product(h, exact(down[e]), f).half()
        d_y = _Known(wr * gr, (2.0 ** -18 + 2 * U) * np.abs(wr * gr)).half()
        d_w.v[t, j] = (gr * y.v).sum(1)
        d_w.e[t, j] = (np.abs(gr) * (y.e + (d + 8) * U * y.top)).sum(1)
        d_h = _product(d_y, _turned(exact(down[e])), d).half()
        d_down = _product(_turned(d_y), _turned(h), len(t)).half()
        # dz at the rounded pre: gate half d_h up silu'(gate), up half d_h silu(gate)
        pg, pu = (_Known(pre.v[:, s_], pre.e[:, s_]) for s_ in (slice(None, f), slice(f, None)))
        slope, sg = OL.derivative("silu", pg.v), OL.activation("silu", pg.v)
        es, eg = 0.5 * pg.e, 1.13 * pg.e
        gate = d_h.v * pu.v * slope
        up_half = d_h.v * sg
        egate = d_h.top * pu.top * (np.abs(slope) + es) - np.abs(gate)
        eup = d_h.top * (np.abs(sg) + eg) - np.abs(up_half)
        own = (16 + 64 * pg.top) * U * d_h.top
        dz = _Known(np.concatenate([gate, up_half], 1), np.concatenate([egate + own * pu.top, eup + own * pg.top], 1))
        dz = dz.half(2.0 ** -39 * dz.top.max())
        d_up = _product(_turned(dz), _turned(xr), len(t)).half()
        dr = _product(dz, _turned(exact(up[e])), 2 * f).half()
        for name, got in (("d_up", d_up), ("d_down", d_down)):
            out[name][0][e], out[name][1][e] = got.v, got.e
        d_rows += [(t[r], dr.v[r], dr.e[r]) for r in range(len(t))]
    size = np.zeros_like(x)
    for t, v, err in d_rows:
        out["dx"][0][t] += v
        out["dx"][1][t] += err
        size[t] += np.abs(v) + err
    dx = _Known(out["dx"][0], out["dx"][1] + (k + 2) * U * size).half()
    out["dx"] = dx.v, dx.e
    # d_logits of a chosen expert: w_j (d_w_j - sum_i w_i d_w_i); of the others 0
    mean = (w * d_w.v).sum(1, keepdims=True)
    v, err = np.zeros_like(a["logits"]), np.zeros_like(a["logits"])
    np.put_along_axis(v, ids.astype(np.int64), w * (d_w.v - mean), 1)
    np.put_along_axis(err, ids.astype(np.int64), w * (d_w.e + (w * d_w.e).sum(1, keepdims=True)), 1)
    out["d_logits"] = v, err + 2.0 ** -17 * d_w.top.max(1, keepdims=True)
    return out


def outside(got, ref):
    """Entries of each gradient that are further off than they can be."""
    return {n: np.abs(got[n] - v) > e for n, (v, e) in ref.items()}


def simulated(a, lost=None):
    """The step with its roundings to fp16 and to fp32 weights (sums in float64), one slot's gradient `lost`."""
    r = lambda v: v.astype(np.float16).astype(np.float64)  # noqa: E731
    x, up, down, g, ids, first = (a[n] for n in ("x", "up", "down", "g", "ids", "first"))
    f = up.shape[1] // 2
    w = OR.weights_of(a["logits"], ids, np.ones(ids.shape, bool), "softmax", True).astype(np.float32).astype(np.float64)
    pos, src, offsets = OS.sort(ids, len(up), first)
    d = {n: np.zeros_like(v) for n, v in (("d_up", up), ("d_down", down))}
    y, d_rows = np.zeros((ids.size, x.shape[1])), np.zeros((ids.size, x.shape[1]))
    rows = OS.permute(x, pos, np.zeros_like(y))
    pieces = [(e, slice(offsets[e], offsets[e + 1])) for e in range(len(up))]
    kept = {}
    for e, s in pieces:
        z = rows[s] @ up[e].T
        kept[e] = r(z), r(OL.apply("swiglu", z))
        y[s] = r(kept[e][1] @ down[e].T)
    d_y, d_w, _ = OS.unpermute_backward(y, pos, w, g, np.zeros_like(y))
    d_y = r(d_y)
    if lost is not None:
        d_y[pos[lost]] = 0
    for e, s in pieces:
        pre, h = kept[e]
        dz = r(OL.dz("swiglu", r(d_y[s] @ down[e]), pre))
        d["d_down"][e], d["d_up"][e], d_rows[s] = r(d_y[s].T @ h), r(dz.T @ rows[s]), r(dz @ up[e])
    d["dx"] = r(OS.unpermute(d_rows, pos)[0])
    d["d_logits"] = OR.route_backward(a["logits"], ids, np.ones(ids.shape, bool), d_w, "softmax", True)
    return d


KINDS = ["signed", "positive"]


@pytest.mark.parametrize("kind", KINDS)
def test_the_formulas_are_differences(kind):
    a = inputs(kind, T=12)
    d = ST.gradients(**a)
    rng = np.random.default_rng(1)
    for arg, name in (("x", "dx"), ("up", "d_up"), ("down", "d_down"), ("logits", "d_logits")):
        for _ in range(4):
            v = rng.standard_normal(a[arg].shape)
            f = [ST.loss(**dict(a, **{arg: a[arg] + s * 1e-5 * v})) for s in (1, -1)]
            assert np.isclose((f[0] - f[1]) / 2e-5, (d[name] * v).sum(), rtol=1e-6, atol=1e-7 * np.abs(d[name] * v).sum()), name
    for name, (v, _) in bounds(a).items():                 # the two ways to the gradients agree
        assert np.allclose(v, d[name], rtol=1e-12, atol=1e-12 * np.abs(v).max()), name


@pytest.mark.parametrize("kind", KINDS)
def test_the_bounds_hold_and_refuse(kind):
    a = inputs(kind)
    ref, got = bounds(a), simulated(a)
    assert not any(o.any() for o in outside(got, ref).values())
    f = a["up"].shape[1] // 2
    # a part that is 5% too small, expert by expert, half by half
    parts = [("dx", np.s_[:]), ("d_logits", np.s_[:])] + [(n, np.s_[e]) for n in ("d_up", "d_down") for e in range(len(a["up"]))]
    parts += [("d_up", np.s_[e, s]) for e in range(len(a["up"])) for s in (slice(None, f), slice(f, None))]
    for name, part in parts:
        bad = {n: v.copy() for n, v in got.items()}
        bad[name][part] *= 0.95
        assert outside(bad, ref)[name][part].any(), (name, part)
    # one slot's row left out of the way back
    t, j = next((t, j) for t, j in np.ndindex(*a["ids"].shape) if 0 <= a["ids"][t, j] - a["first"] < len(a["up"]))
    e = a["ids"][t, j] - a["first"]
    far = outside(simulated(a, lost=(t, j)), ref)
    assert far["dx"][t].any() and far["d_up"][e].any() and far["d_down"][e].any()
    # halves or experts in each other's place
    for name, turn in (("d_up", lambda v: np.roll(v, f, 1)), ("d_up", lambda v: np.roll(v, 1, 0)), ("d_down", lambda v: np.roll(v, 1, 0)),
                       ("dx", lambda v: np.roll(v, 1, 0)), ("d_logits", lambda v: np.roll(v, 1, 1))):
        assert outside(dict(got, **{name: turn(got[name])}), ref)[name].mean() > 0.5 * (np.abs(got[name]) > 0).mean(), name


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T", [("signed", 48), ("positive", 48), ("signed", 1), ("positive", 300)])
def test_training_step(kind, T):
    import torch

    import moe_expert_tile_amd as m
    a = inputs(kind, T=T, seed=T)
    ref = bounds(a)
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    on = lambda n, dtype=f16: torch.from_numpy(a[n]).to(dtype).cuda()  # noqa: E731
    full = lambda *s, dtype=f16: torch.full(s, 9, dtype=dtype, device="cuda")  # noqa: E731
    x, up, down, g, logits = on("x"), on("up"), on("down"), on("g"), on("logits", f32)
    E, (d, f), k = len(up), down.shape[1:], a["ids"].shape[1]
    ids, w = full(T, k, dtype=i32), full(T, k, dtype=f32)
    m.moe_route(logits, ids, w, renorm=True)
    assert np.array_equal(ids.cpu().numpy(), a["ids"])
    pos, offsets = full(T, k, dtype=i32), full(E + 1, dtype=i32)
    m.moe_sort(ids, pos, offsets, first=a["first"])
    rows, pre, h, y, out = full(T * k, d), full(T * k, 2 * f), full(T * k, f), full(T * k, d), full(T, d)
    m.moe_permute(x, pos, rows)
    off = offsets.tolist()
    pieces = [(e, slice(off[e], off[e + 1])) for e in range(E)]        # experts without rows too
    for e, s in pieces:
        m.moe_linear(rows[s], up[e], h[s], pre=pre[s], act=m.ACT_SWIGLU)
        m.moe_linear(h[s], down[e], y[s])
    m.moe_unpermute(y, pos, out, topk_w=w)
    d_y, d_w, d_h, d_rows = full(T * k, d), full(T, k, dtype=f32), full(T * k, f), full(T * k, d)
    dx, d_up, d_down, d_logits = (torch.full_like(t, 9) for t in (x, up, down, logits))
    m.moe_unpermute_backward(pos, g, y, w, d_y, d_w)
    for e, s in pieces:
        m.moe_linear_backward(h[s], down[e], d_y[s], dx=d_h[s], dw=d_down[e])
        m.moe_linear_backward(rows[s], up[e], d_h[s], dx=d_rows[s], dw=d_up[e], pre=pre[s], act=m.ACT_SWIGLU)
    m.moe_permute_backward(d_rows, pos, dx)
    m.moe_route_backward(logits, ids, w, d_w, d_logits, renorm=True)
    torch.cuda.synchronize()
    got = {"dx": dx, "d_up": d_up, "d_down": d_down, "d_logits": d_logits}
    for name, far in outside({n: t.double().cpu().numpy() for n, t in got.items()}, ref).items():
        assert not far.any(), (name, np.argwhere(far)[:4].tolist())
