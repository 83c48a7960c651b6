"""Refusals of the calls on rows sorted by expert, without a GPU: bad sizes,
pointers and tensors are errors before any HIP call.  And the oracle's own
pins."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import rows as OR

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_tile_amd", "libmoe.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")

GOOD = 1 << 20   # never dereferenced: validation fails first


def _m():
    import moe_expert_tile_amd as m
    return m


@built
@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=(1 << 26) + 1), dict(top_k=0), dict(top_k=33), dict(experts=0), dict(experts=1025),
    dict(tokens=1 << 26, top_k=32), dict(first=-1), dict(first=2 ** 31 - 15), dict(ids=0), dict(ids=GOOD + 2), dict(pos=0), dict(pos=GOOD + 1),
    dict(src=GOOD + 2), dict(offsets=0), dict(offsets=GOOD + 2), dict(ws=GOOD + 128), dict(tokens=32768, ws=0)])
def test_bad_sorts_are_rejected(bad):
    m = _m()
    a = dict(tokens=4, top_k=2, experts=16, first=0, ids=GOOD, pos=GOOD, src=None, offsets=GOOD, ws=GOOD)
    a.update(bad)
    assert m._lib.moe_sort(*a.values(), 0) == m.MOE_EINVAL


@built
def test_sort_workspace_sizes():
    m = _m()
    assert m.moe_sort_sizes(1, 1, 1) == 0 and m.moe_sort_sizes(0, 8, 64) == 0
    for T, k, E in ((32768, 8, 256), ((1 << 26) - 1, 31, 1024), (1 << 26, 31, 8)):
        assert 0 < m.moe_sort_sizes(T, k, E) <= 256 * 4 * E
    with pytest.raises(m.MoEError):
        m.moe_sort_sizes(1 << 26, 32, 8)
    assert m._lib.moe_sort_sizes(4, 2, 16, None) == m.MOE_EINVAL


BAD_DESC = [dict(tokens=-1), dict(tokens=(1 << 26) + 1), dict(rows=-1), dict(rows=1 << 31), dict(top_k=0),
            dict(top_k=33), dict(cols=0), dict(cols=(1 << 20) + 1), dict(dtype=3), dict(dtype=-1), dict(pad=1),
            dict(ld_x=31), dict(ld_rows=-32), dict(ld_d_rows=16), dict(ld_x=(1 << 21) + 1), dict(ld_rows=(1 << 21) + 1)]


@built
def test_bad_row_calls_are_rejected():
    m = _m()

    def desc(**kw):
        return ctypes.byref(m.moe_rows_desc(**dict(dict(tokens=4, rows=8, top_k=2, cols=32, dtype=0), **kw)))

    calls = {"moe_permute": 3, "moe_permute_backward": 3, "moe_unpermute": 4, "moe_unpermute_backward": 6}
    for name, n in calls.items():
        fn = getattr(m._lib, name)
        for bad in BAD_DESC:
            assert fn(desc(**bad), *[GOOD] * n, 0) == m.MOE_EINVAL, (name, bad)
        assert fn(None, *[GOOD] * n, 0) == m.MOE_EINVAL
        for i in range(n):
            a = [GOOD] * n
            a[i] = GOOD + 1                       # no element's address
            assert fn(desc(), *a, 0) == m.MOE_EINVAL, (name, i)
            a[i] = GOOD + 2
            assert fn(desc(dtype=2), *a, 0) == m.MOE_EINVAL, (name, i)
    for name, n, needed in (("moe_permute", 3, (0, 1, 2)), ("moe_permute_backward", 3, (0, 1, 2)),
                            ("moe_unpermute", 4, (0, 1, 3)), ("moe_unpermute_backward", 6, (0, 1, 3))):
        for i in needed:
            a = [GOOD] * n
            a[i] = None
            assert getattr(m._lib, name)(desc(), *a, 0) == m.MOE_EINVAL, (name, i)
    assert m._lib.moe_unpermute_backward(desc(), GOOD, GOOD, GOOD, GOOD, None, None, 0) == m.MOE_EINVAL


@built
def test_empty_gradients_are_no_refusal():
    """Without tokens or without rows a gradient that was asked for may have no
    address; with both, a call for neither is refused."""
    m = _m()

    def call(tokens, rows, d_rows, d_topk_w):
        d = m.moe_rows_desc(tokens=tokens, rows=rows, top_k=2, cols=32, dtype=0)
        return m._lib.moe_unpermute_backward(ctypes.byref(d), GOOD if rows and d_topk_w else None, GOOD if tokens else None, None,
                                             GOOD if tokens else None, d_rows, d_topk_w, 0)

    for sizes in ((3, 0), (0, 4), (0, 0)):       # nothing to write: no launch, and without a GPU no device
        assert call(*sizes, None, None) in (m.MOE_OK, m.MOE_EHIP, m.MOE_EUNSUPPORTED), sizes
    assert call(3, 4, None, None) == m.MOE_EINVAL
    pos, g, rows = torch.zeros(0, 2, dtype=torch.int32), torch.zeros(0, 32), torch.zeros(0, 32)
    with pytest.raises(m.MoEError) as ei:
        m.moe_unpermute_backward(pos, g, rows)
    assert ei.value.status == m.MOE_EINVAL and "neither d_rows nor d_topk_w" in str(ei.value)


@built
def test_bad_row_tensors_are_rejected():
    m = _m()
    ids, pos, offsets = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    for a, kw in (((ids.long(), pos, offsets), {}), ((ids[0], pos, offsets), {}), ((ids, pos[:3], offsets), {}),
                  ((ids, pos.long(), offsets), {}), ((ids, pos, offsets.float()), {}), ((ids, pos, offsets[:0]), {}),
                  ((ids, pos, offsets[:1]), {}), ((ids, pos, offsets.view(3, 3)), {}),
                  ((ids.t().contiguous().t(), pos, offsets), {}), ((ids, pos.t().contiguous().t(), offsets), {}),
                  ((ids, pos, offsets), dict(src=torch.zeros(7, dtype=torch.int32))),
                  ((ids, pos, offsets), dict(src=torch.zeros(8))), ((ids, pos, offsets), dict(first=-1)),
                  ((ids, pos, offsets), dict(ws=torch.zeros(16)[::2])), ((ids, pos, offsets), {})):
        with pytest.raises(m.MoEError) as ei:      # the last one is sound but for its device
            m.moe_sort(*a, **kw)
        assert ei.value.status == m.MOE_EINVAL
    x, rows, w = torch.zeros(4, 32), torch.zeros(8, 32), torch.zeros(4, 2)
    for bad in (dict(x=x.double()), dict(x=x[:3]), dict(x=x.half()), dict(x=x[:, :31]), dict(x=x.t().contiguous().t()),
                dict(x=x[:1].expand(4, 32)), dict(rows=rows[0]), dict(rows=rows[:1].expand(8, 32)),
                dict(pos=pos.long()), dict(pos=pos[:, :1]), dict(pos=pos[:3]), dict()):
        a = dict(dict(x=x, pos=pos, rows=rows), **bad)
        for call in (lambda: m.moe_permute(a["x"], a["pos"], a["rows"]),
                     lambda: m.moe_permute_backward(a["rows"], a["pos"], a["x"]),
                     lambda: m.moe_unpermute(a["rows"], a["pos"], a["x"], topk_w=w),
                     lambda: m.moe_unpermute_backward(a["pos"], a["x"], a["rows"], w, a["rows"], w)):
            with pytest.raises(m.MoEError) as ei:
                call()
            assert ei.value.status == m.MOE_EINVAL, bad
    for call in (lambda: m.moe_unpermute(rows, pos, x, topk_w=w.double()),
                 lambda: m.moe_unpermute(rows, pos, x, topk_w=w[:, :1]),
                 lambda: m.moe_unpermute_backward(pos, x, rows, w),
                 lambda: m.moe_unpermute_backward(pos, x, topk_w=w, d_topk_w=w),
                 lambda: m.moe_unpermute_backward(pos, x, rows[:7], w, d_rows=rows),
                 lambda: m.moe_unpermute_backward(pos, x, rows, w, d_topk_w=w.bfloat16())):
        with pytest.raises(m.MoEError) as ei:
            call()
        assert ei.value.status == m.MOE_EINVAL


def test_the_oracle_sorts():
    ids = np.array([[3, 1], [1, 3], [9, 2], [2, -1]], np.int32)
    pos, src, offsets = OR.sort(ids, 4)
    assert pos.tolist() == [[4, 0], [1, 5], [-1, 2], [3, -1]]
    assert src.tolist() == [1, 2, 5, 6, 0, 3] and offsets.tolist() == [0, 0, 2, 4, 6]
    pos, src, offsets = OR.sort(ids, 2, first=2)
    assert pos.tolist() == [[2, -1], [-1, 3], [-1, 0], [1, -1]] and offsets.tolist() == [0, 2, 4]


def test_the_oracle_rows_are_each_others_gradients():
    rng = np.random.default_rng(0)
    ids = rng.integers(0, 5, (6, 3)).astype(np.int32)
    pos, src, _ = OR.sort(ids, 4)
    x, w, y = rng.standard_normal((6, 8)), rng.standard_normal((6, 3)), rng.standard_normal((18, 8))
    rows = OR.permute(x, pos, np.zeros((18, 8)))
    assert np.array_equal(rows[:len(src)], x[src // 3]) and not rows[len(src):].any()
    # <permute x, y> = <x, sum of y's rows>
    y[len(src):] = 0
    assert np.isclose((rows * y).sum(), (x * OR.unpermute(y, pos)[0]).sum())
    g = rng.standard_normal((6, 8))
    d_rows, d_w, _ = OR.unpermute_backward(y, pos, w, g, np.zeros_like(y))
    h = 1e-6
    for _ in range(3):
        vy, vw = rng.standard_normal(y.shape), rng.standard_normal(w.shape)
        f = [(g * OR.unpermute(y + s * h * vy, pos, w + s * h * vw)[0]).sum() for s in (1, -1)]
        assert np.isclose((f[0] - f[1]) / (2 * h), (d_rows * vy).sum() + (d_w * vw).sum(), rtol=1e-6)
