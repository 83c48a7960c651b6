"""Refusals of the calls on microscaled 4-bit rows, without a GPU: bad sizes,
pointers and tensors are errors before any HIP call.  And the oracle's own
pins."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import mx as OM

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_tile_amd", "libmoe.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")

GOOD = 1 << 20   # never dereferenced: validation fails first


def _m():
    import moe_expert_tile_amd as m
    return m


@built
@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=1 << 31), dict(depth=0), dict(depth=48), dict(depth=(1 << 20) + 32), dict(dtype=3),
    dict(dtype=-1), dict(x=0), dict(x=GOOD + 1), dict(x=GOOD + 2, dtype=2), dict(ld_x=63), dict(ld_x=(1 << 21) + 1),
    dict(q=0), dict(q=GOOD + 8), dict(ld_q=16), dict(ld_q=40), dict(ld_q=1 << 22), dict(scale=0), dict(ld_s=1),
    dict(ld_s=-2), dict(ld_s=(1 << 21) + 1)])
def test_bad_quantisations_are_rejected(bad):
    m = _m()
    a = dict(rows=4, depth=64, x=GOOD, dtype=0, ld_x=0, q=GOOD, ld_q=0, scale=GOOD + 1, ld_s=0)
    a.update(bad)
    assert m._lib.moe_mx_quantize(*a.values(), 0) == m.MOE_EINVAL
    assert m._lib.moe_mx_dequantize(a["rows"], a["depth"], a["q"], a["ld_q"], a["scale"], a["ld_s"], a["x"], a["dtype"],
                                    a["ld_x"], 0) == m.MOE_EINVAL


BAD_DESC = [dict(rows=-1), dict(rows=(1 << 26) + 1), dict(experts=0), dict(experts=1025), dict(cols=0),
            dict(cols=(1 << 20) + 1), dict(depth=0), dict(depth=80), dict(depth=(1 << 20) + 32), dict(dtype=2),
            dict(dtype=4), dict(out_dtype=1), dict(out_dtype=3), dict(dtype=1, out_dtype=0), dict(dtype=3, out_dtype=3),
            dict(act=6), dict(act=-1), dict(ld_x=68), dict(ld_x=56), dict(dtype=3, ld_x=40), dict(ld_x_scale=1),
            dict(ld_w=16), dict(ld_w=40), dict(ld_w_scale=1), dict(ld_out=31), dict(ld_w=1 << 22), dict(expert_w=24),
            dict(expert_w=-16), dict(expert_w_scale=-1), dict(expert_w=1 << 43)]


@built
@pytest.mark.parametrize("bad", BAD_DESC)
def test_bad_product_sizes_are_rejected(bad):
    m = _m()
    d = m.moe_mx_linear_desc(**dict(dict(rows=4, experts=2, cols=32, depth=64, dtype=0, out_dtype=0, act=0), **bad))
    assert m._lib.moe_mx_linear(ctypes.byref(d), *[GOOD] * 7, 0) == m.MOE_EINVAL


@built
def test_bad_product_pointers_are_rejected():
    m = _m()

    def call(x=GOOD, xs=GOOD, w=GOOD, ws=GOOD, offsets=GOOD, bias=GOOD, out=GOOD, **kw):
        d = m.moe_mx_linear_desc(**dict(dict(rows=4, experts=2, cols=32, depth=64, dtype=0, out_dtype=0), **kw))
        return m._lib.moe_mx_linear(ctypes.byref(d), x, xs, w, ws, offsets, bias, out, 0)

    for bad in (dict(x=None), dict(x=GOOD + 8), dict(w=None), dict(w=GOOD + 8), dict(ws=None), dict(offsets=None),
                dict(offsets=GOOD + 2), dict(bias=GOOD + 1), dict(out=None), dict(out=GOOD + 1),
                dict(out_dtype=2, out=GOOD + 2), dict(out_dtype=2, bias=GOOD + 2), dict(dtype=3, xs=None)):
        assert call(**bad) == m.MOE_EINVAL, bad
    assert m._lib.moe_mx_linear(None, *[GOOD] * 7, 0) == m.MOE_EINVAL


@built
def test_bad_tensors_are_rejected():
    m = _m()
    u8, bf = torch.uint8, torch.bfloat16
    x, q, s = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 32, dtype=u8), torch.zeros(4, 2, dtype=u8)
    for bad in (dict(x=x.double()), dict(x=x[:3]), dict(x=x[:, :48]), dict(x=x[:, :0]), dict(x=x[0]), dict(q=q[:, :31]), dict(q=q.int()),
                dict(q=q[0]), dict(s=s[:, :1]), dict(s=s.float()), dict(s=s[:1].expand(4, 2)),
                dict(q=q.t().contiguous().t()), dict()):
        a = dict(dict(x=x, q=q, s=s), **bad)      # the last one is sound but for its device
        for call in (lambda: m.moe_mx_quantize(a["x"], a["q"], a["s"]), lambda: m.moe_mx_dequantize(a["q"], a["s"], a["x"])):
            with pytest.raises(m.MoEError) as ei:
                call()
            assert ei.value.status == m.MOE_EINVAL, bad
    w, ws, out, off = torch.zeros(2, 32, 32, dtype=u8), torch.zeros(2, 32, 2, dtype=u8), torch.zeros(4, 32, dtype=bf), torch.zeros(3, dtype=torch.int32)
    good = dict(x=x, w=w, w_scale=ws, out=out, offsets=off)
    for bad in (dict(x=x.float()), dict(x=x.half()), dict(x=x[:3]), dict(x=x[:, :32]), dict(x=x[:, :40]), dict(w=w[:, :31]), dict(w=w[0]),
                dict(w=w.int()), dict(w=w[:1].expand(2, 32, 32)), dict(w=w.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(w_scale=ws[:1]), dict(w_scale=ws[:, :, :1]), dict(w_scale=ws[0]), dict(out=out.half()), dict(out=out[0]),
                dict(offsets=None), dict(offsets=off[:2]), dict(offsets=off.long()), dict(bias=torch.zeros(2, 32)),
                dict(bias=torch.zeros(32, dtype=bf)), dict(act=m.ACT_SWIGLU), dict(act=9), dict(x=q, x_scale=s[:, :1]),
                dict(x=q.int(), x_scale=s), dict(x=q), dict(x=q, x_scale=s, out=out.double()), dict(x=x, x_scale=s), dict()):
        with pytest.raises(m.MoEError) as ei:
            m.moe_mx_linear(**dict(good, **bad))
        assert ei.value.status == m.MOE_EINVAL, bad


def test_the_oracle_rounds_to_the_next_element():
    for y, want in ((0, 0), (0.25, 0), (0.26, 0.5), (0.75, 1), (1.25, 1), (1.3, 1.5), (1.75, 2), (2.5, 2), (2.51, 3), (3.5, 4),
                    (5, 4), (5.01, 6), (7.9, 6), (-0.2, -0.0), (-2.5, -2), (-5.5, -6)):
        got = OM.ELEMENTS[OM.element(y)]
        assert got == want and np.signbit(got) == np.signbit(want), (y, got)


def test_the_oracle_blocks():
    x = np.zeros((1, 96))
    x[0, :32] = np.linspace(-7.99, 7.99, 32)       # largest below 8: scale 1
    x[0, 33] = 2.0 ** -130                         # scale 2^-127: far below its smallest element
    x[0, 70] = np.inf
    q, s = OM.quantize(x)
    assert s.tolist() == [[127, 0, 255]]
    v = OM.values(q, s)
    assert set(np.abs(v[0, :32])) <= set(np.abs(OM.ELEMENTS)) and v[0, 31] == 6 and v[0, 0] == -6
    assert (v[0, 32:64] == 0).all() and np.isnan(v[0, 64:]).all()
    # within half a step of the range below 6, at most 2 above it
    assert np.all(np.abs(v[0, :32] - x[0, :32]) <= np.where(np.abs(x[0, :32]) < 6, 1.0, 2.0))
    # what stands for itself stays itself
    again = OM.quantize(v[:, :64])
    assert np.array_equal(OM.values(*again), v[:, :64])
