"""Refusals of the routing, dense-product and scale-gradient calls, without a
GPU: bad sizes, options, pointers and tensors are errors before any HIP call."""
import ctypes
import os

import pytest
import torch

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_tile_amd", "libmoe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")

GOOD = 1 << 20   # never dereferenced: validation fails first


def _m():
    import moe_expert_tile_amd as m
    return m


def _route(m, tokens=4, experts=16, top_k=2, logits=GOOD, dtype=0, ld=0, bias=None, opts=None, ids=GOOD, w=GOOD):
    o = m.moe_route_opts(**opts) if opts is not None else None
    return m._lib.moe_route(tokens, experts, top_k, logits, dtype, ld, bias, ctypes.byref(o) if o else None, ids, w, 0)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=(1 << 26) + 1), dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=17),
    dict(experts=64, top_k=33), dict(dtype=3), dict(dtype=-1), dict(ld=15), dict(ld=-16), dict(ld=(1 << 21) + 1),
    dict(logits=0), dict(logits=GOOD + 1), dict(dtype=2, logits=GOOD + 2), dict(ids=0), dict(ids=GOOD + 2), dict(w=0),
    dict(w=GOOD + 1), dict(bias=GOOD + 2),
    dict(opts=dict(score=2)), dict(opts=dict(score=-1)), dict(opts=dict(scale=-1.0)),
    dict(opts=dict(scale=float("nan"))), dict(opts=dict(scale=float("inf"))),
    dict(opts=dict(n_group=3)), dict(opts=dict(n_group=-1)), dict(experts=1024, opts=dict(n_group=128)),
    dict(opts=dict(n_group=4, topk_group=5)), dict(opts=dict(n_group=4, topk_group=-1)),
    dict(opts=dict(n_group=4, group_score=2)), dict(opts=dict(n_group=16, group_score=1)),
    dict(top_k=5, opts=dict(n_group=4, topk_group=1)),
])
def test_bad_route_calls_are_rejected(bad):
    m = _m()
    assert _route(m, **bad) == m.MOE_EINVAL


def test_bad_route_backward_calls_are_rejected():
    m = _m()

    def call(tokens=4, experts=16, top_k=2, logits=GOOD, dtype=0, ld=0, ids=GOOD, w=GOOD, dw=GOOD, opts=None, dz=GOOD,
             ld_d=0):
        o = m.moe_route_opts(**opts) if opts is not None else None
        return m._lib.moe_route_backward(tokens, experts, top_k, logits, dtype, ld, ids, w, dw,
                                         ctypes.byref(o) if o else None, dz, ld_d, 0)

    for bad in (dict(tokens=-1), dict(experts=0), dict(top_k=0), dict(top_k=17), dict(dtype=5), dict(ld=3),
                dict(ld_d=15), dict(ld_d=-1), dict(logits=0), dict(ids=0), dict(w=0), dict(dw=0), dict(dz=0),
                dict(ids=GOOD + 1), dict(dw=GOOD + 2), dict(dz=GOOD + 1), dict(opts=dict(score=7)),
                dict(opts=dict(scale=-2.0))):
        assert call(**bad) == m.MOE_EINVAL, bad


def _desc(m, **kw):
    base = dict(rows=4, cols=32, depth=64, dtype=0, out_dtype=0, act=0, pad=0)
    base.update(kw)
    return m.moe_linear_desc(**base)


BAD_DESC = [dict(rows=-1), dict(rows=(1 << 21) + 1), dict(cols=0), dict(cols=(1 << 20) + 1), dict(depth=0),
            dict(depth=60), dict(depth=(1 << 20) + 8), dict(dtype=2), dict(dtype=-1), dict(out_dtype=1),
            dict(out_dtype=3), dict(dtype=1, out_dtype=0), dict(act=6), dict(act=-1), dict(pad=1), dict(ld_x=56),
            dict(ld_x=68), dict(ld_w=-64), dict(ld_w=66), dict(ld_residual=31), dict(ld_pre=31), dict(ld_out=16),
            dict(act=5, ld_pre=63), dict(ld_dx=63), dict(ld_dw=63), dict(ld_x=(1 << 21) + 8)]


@pytest.mark.parametrize("bad", BAD_DESC)
def test_bad_linear_sizes_are_rejected(bad):
    m = _m()
    d = _desc(m, **bad)
    with pytest.raises(m.MoEError) as ei:
        m.moe_linear_sizes(d)
    assert ei.value.status == m.MOE_EINVAL
    assert m._lib.moe_linear(ctypes.byref(d), GOOD, GOOD, None, None, None, GOOD, GOOD, 0) == m.MOE_EINVAL
    assert m._lib.moe_linear_backward(ctypes.byref(d), GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, 0) == m.MOE_EINVAL


def test_bad_linear_pointers_are_rejected():
    m = _m()

    def call(x=GOOD, w=GOOD, bias=None, res=None, pre=None, out=GOOD, ws=GOOD, **kw):
        return m._lib.moe_linear(ctypes.byref(_desc(m, **kw)), x, w, bias, res, pre, out, ws, 0)

    for bad in (dict(x=0), dict(w=0), dict(out=0), dict(x=GOOD + 8), dict(w=GOOD + 2), dict(out=GOOD + 1),
                dict(bias=GOOD + 1), dict(res=GOOD + 1), dict(pre=GOOD + 1), dict(ws=GOOD + 128),
                dict(out_dtype=2, out=GOOD + 2), dict(out_dtype=2, res=GOOD + 2),
                dict(res=GOOD, ld_residual=64)):     # in place with another pitch
        assert call(**bad) == m.MOE_EINVAL, bad
    assert m._lib.moe_linear(None, GOOD, GOOD, None, None, None, GOOD, GOOD, 0) == m.MOE_EINVAL
    split = dict(rows=128, cols=64, depth=8192)      # few tiles, long sums: split along K
    assert m.moe_linear_sizes(_desc(m, **split))["forward_bytes"] > 0
    assert call(ws=0, **split) == m.MOE_EINVAL

    def back(x=GOOD, w=GOOD, pre=GOOD, d_out=GOOD, dx=GOOD, dw=GOOD, db=GOOD, ws=GOOD, **kw):
        return m._lib.moe_linear_backward(ctypes.byref(_desc(m, **kw)), x, w, pre, d_out, dx, dw, db, ws, 0)

    for bad in (dict(dx=0, dw=0, db=0), dict(d_out=0), dict(x=0), dict(w=0), dict(act=2, pre=0), dict(ws=0),
                dict(ws=GOOD + 16), dict(x=GOOD + 8), dict(dx=GOOD + 1), dict(dw=GOOD + 1), dict(db=GOOD + 1),
                dict(out_dtype=2, d_out=GOOD + 2)):
        assert back(**bad) == m.MOE_EINVAL, bad


def test_bad_scale_backward_calls_are_rejected():
    m = _m()
    s = m.Shape(4, 0, 2, 2, 512, 1024, 64, [256] * 4, 500)
    ok = dict(plan=GOOD, recv=GOOD, w=GOOD, g=GOOD, dr=GOOD, dw=GOOD)
    for bad in (dict(plan=0), dict(plan=GOOD + 16), dict(recv=0), dict(recv=GOOD + 8), dict(w=0), dict(w=GOOD + 2),
                dict(g=0), dict(g=GOOD + 8), dict(dr=0, dw=0), dict(dr=GOOD + 8), dict(dw=GOOD + 2)):
        a = dict(ok, **bad)
        with pytest.raises(m.MoEError) as ei:
            m.moe_scale_backward(s, a["plan"], a["recv"], a["w"], a["g"], a["dr"] or None, a["dw"] or None, stream=0)
        assert ei.value.status == m.MOE_EINVAL, bad


def test_bad_tensors_are_rejected():
    m = _m()
    z, ids, w = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    g = torch.zeros(4, 16)
    route = [(z.double(), ids, w), (z[0], ids, w), (z, ids.long(), w), (z, ids[:3], w), (z, ids, w[:, :1]),
             (z, ids.t().contiguous().t(), w), (z.t().contiguous().t(), ids, w), (z, ids[0], w), (z, ids, w)]
    for a in route:      # the last one is sound but for its device
        with pytest.raises(m.MoEError) as ei:
            m.moe_route(*a)
        assert ei.value.status == m.MOE_EINVAL
        with pytest.raises(m.MoEError):
            m.moe_route_backward(a[0], a[1], a[2], w, g)
    x, wt, out = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 64), (32, 64), (4, 32)))
    for kw in (dict(x=x.float()), dict(x=x.half()), dict(w=wt[:31]), dict(w=wt[:, :32]), dict(out=out.half()),
               dict(out=out[:3]), dict(x=x.t().contiguous().t()), dict(bias=torch.zeros(32)),
               dict(bias=torch.zeros(31, dtype=torch.bfloat16)), dict(residual=out.float()), dict(pre=out.float()),
               dict(act=m.ACT_SWIGLU), dict(act=9), dict(x=x[0]), dict(x=x[:, :60], w=wt[:, :60])):
        a = dict(dict(x=x, w=wt, out=out), **kw)
        with pytest.raises(m.MoEError) as ei:
            m.moe_linear(**a)
        assert ei.value.status == m.MOE_EINVAL, kw
    for kw in (dict(dx=x.float()), dict(dw=wt[:3]), dict(dbias=torch.zeros(32)), dict(pre=x)):
        with pytest.raises(m.MoEError):
            m.moe_linear_backward(x, wt, out, **kw)


def test_linear_workspace_sizes():
    """Few rows and many tiles need no forward workspace; a split product one
    fp32 copy of its sums per split."""
    m = _m()
    assert m.moe_linear_sizes(_desc(m, rows=1, cols=7168, depth=2048))["forward_bytes"] == 0
    assert m.moe_linear_sizes(_desc(m, rows=8192, cols=4096, depth=4096))["forward_bytes"] == 0
    z = m.moe_linear_sizes(_desc(m, rows=128, cols=64, depth=8192))
    assert z["forward_bytes"] % (128 * 64 * 4) == 0 and z["backward_bytes"] > 0
    for kw in (dict(rows=0), dict(rows=0, cols=1, depth=8, act=5), dict(rows=1), dict(rows=1 << 21)):
        z = m.moe_linear_sizes(_desc(m, **kw))
        assert z["backward_bytes"] > 0 and z["forward_bytes"] == 0, kw
