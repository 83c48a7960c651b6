"""Rows sorted by expert on the GPU: sort, tokens to rows, weighted sum back and
the gradients against the float64 oracle, from one token to batches of many
workgroups, with slots and tokens that have no row, odd columns and pitches."""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import rows as OR

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11), "f32": (torch.float32, 2.0 ** -24)}


def _m():
    import moe_expert_tile_amd as m
    return m


def _np(t):
    return t.detach().double().cpu().numpy()


def _sorted(ids, E, first=0):
    m = _m()
    T, k = ids.shape
    ids = torch.from_numpy(ids).cuda()
    pos = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    src, offsets = torch.full((T * k,), 77, dtype=torch.int32, device="cuda"), torch.full((E + 1,), 77, dtype=torch.int32, device="cuda")
    m.moe_sort(ids, pos, offsets, src=src, first=first)
    return pos, src, offsets


SORTS = [(1, 1, 1, 0, 1), (1, 8, 8, 0, 8), (3, 2, 1, 1, 3), (64, 8, 128, 0, 128), (65, 7, 60, 0, 60), (511, 8, 16, 32, 64),
         (512, 8, 1024, 0, 1024), (513, 8, 256, 0, 256), (700, 32, 1000, 0, 1024), (4097, 1, 3, 0, 3),
         (9000, 6, 33, 5, 40), (33000, 8, 257, 0, 256), (140000, 8, 64, 0, 64)]


@pytest.mark.parametrize("T,k,E,first,total", SORTS)
def test_sort(T, k, E, first, total):
    say(f"[sort] T={T} k={k} E={E} first={first} of {total}")
    rng = np.random.default_rng(T + E)
    # uneven experts, some ids of no expert at all
    ids = np.minimum((rng.random((T, k)) ** 2 * total).astype(np.int64), total - 1)
    odd = rng.random((T, k)) < 0.02
    ids = np.where(odd, rng.choice([-1, -2 ** 31, 2 ** 31 - 1, total, first - 1], (T, k)), ids).astype(np.int32)
    pos, src, offsets = _sorted(ids, E, first)
    order = np.argsort(np.where((ids >= first) & (ids < first + E), ids.astype(np.int64), 2 ** 40).reshape(-1), kind="stable")
    want = OR.sort(ids, E, first) if T < 1000 else None
    got = [t.cpu().numpy() for t in (pos, src, offsets)]
    R = got[2][E]
    assert R == ((ids >= first) & (ids.astype(np.int64) < first + E)).sum()
    assert np.array_equal(got[1][:R], order[:R]) and (got[1][R:] == 77).all()
    if want is not None:
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1][:R], want[1]) and np.array_equal(got[2], want[2])
    else:
        inverse = np.full(T * k, -1)
        inverse[order[:R]] = np.arange(R)
        assert np.array_equal(got[0].reshape(-1), inverse)
        local = ids.reshape(-1).astype(np.int64) - first
        assert np.array_equal(got[2], np.concatenate([[0], np.cumsum(np.bincount(local[(local >= 0) & (local < E)], minlength=E))]))


@pytest.mark.parametrize("T", [5, 20000])
def test_sort_of_one_expert_and_of_none(T):
    for e in (3, 99):
        pos, src, offsets = _sorted(np.full((T, 4), e, np.int32), 8)
        if e == 3:
            assert torch.equal(pos.view(-1), torch.arange(4 * T, device="cuda")) and torch.equal(src, pos.view(-1))
            assert offsets.tolist() == [0] * 4 + [4 * T] * 5
        else:
            assert bool((pos == -1).all()) and bool((src == 77).all()) and offsets.tolist() == [0] * 9


def test_sort_of_no_tokens_and_without_src():
    m = _m()
    e = torch.empty(0, 8, dtype=torch.int32, device="cuda")
    offsets = torch.full((5,), 77, dtype=torch.int32, device="cuda")
    m.moe_sort(e, torch.empty_like(e), offsets)
    assert offsets.tolist() == [0] * 5
    ids = torch.randint(0, 4, (1000, 8), dtype=torch.int32, device="cuda")
    pos, pos2 = torch.empty_like(ids), torch.empty_like(ids)
    ws = torch.full((m.moe_sort_sizes(1000, 8, 4),), 255, dtype=torch.uint8, device="cuda")
    m.moe_sort(ids, pos, offsets, src=torch.empty(8000, dtype=torch.int32, device="cuda"))
    m.moe_sort(ids, pos2, offsets, ws=ws)
    assert torch.equal(pos, pos2)


# tokens, slots, columns, pitch beyond them, offset of the first element, dropped slots, spare rows
ROWS = [(1, 1, 1, 0, 0, 0.0, 0), (1, 8, 7168, 0, 0, 0.0, 0), (3, 3, 7, 0, 1, 0.3, 2), (64, 8, 2048, 0, 0, 0.0, 0),
        (65, 6, 1001, 0, 0, 0.2, 5), (33, 2, 513, 3, 1, 0.0, 0), (40, 4, 256, 8, 8, 0.5, 3), (17, 32, 40, 0, 3, 0.1, 0),
        (200, 5, 4104, 0, 0, 1.0, 4), (600, 3, 2500, 4, 0, 0.1, 1), (2100, 2, 64, 0, 0, 0.0, 0)]


def _buffer(gen, rows, cols, more, at, dtype, fill=None):
    """A [rows, cols] matrix of that pitch inside a larger buffer, and the buffer."""
    whole = torch.randn(rows * (cols + more) + at + 16, generator=gen, device="cuda").to(dtype)
    if fill is not None:
        whole.fill_(fill)
    return whole[at:at + rows * (cols + more)].view(rows, cols + more)[:, :cols], whole


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,k,d,more,at,dropped,spare", ROWS)
def test_rows_and_gradients(T, k, d, more, at, dropped, spare, dtype):
    say(f"[rows] T={T} k={k} d={d} +{more} at {at} dropped={dropped} {dtype}")
    m = _m()
    t, half = TYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    rng = np.random.default_rng(T + d)
    ids = rng.integers(0, 6, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < dropped] = 6
    pos, _, offsets = _sorted(ids, 6)
    R = int(offsets[6])
    held = _np(pos).astype(np.int64)
    # a place outside the buffer counts as none
    for p in (R + spare, 2 ** 31 - 1, -2 ** 31):
        bad = rng.integers(0, T * k)
        if held.reshape(-1)[bad] >= 0 and T > 10:
            held.reshape(-1)[bad] = p
    pos = torch.from_numpy(held.astype(np.int32)).cuda()
    x, _ = _buffer(gen, T, d, more, at, t)
    rows, rows_all = _buffer(gen, R + spare, d, more, at, t, 9.0)
    want = OR.permute(_np(x), held, _np(rows))
    m.moe_permute(x, pos, rows)
    assert np.array_equal(_np(rows), want)                      # a copy; rows without a slot as they were
    inside = torch.zeros_like(rows_all, dtype=torch.bool)
    inside[at:at + rows.shape[0] * (d + more)].view(-1, d + more)[:, :d] = True
    assert bool((rows_all[~inside] == 9).all())                 # and all around them
    y, _ = _buffer(gen, R + spare, d, more, at, t)
    w = torch.randn(T, k, generator=gen, device="cuda")
    w[0, 0] = 0
    w[torch.from_numpy((held < 0) | (held >= R + spare)).cuda()] = float("nan")     # weights of no row do not matter
    for weights in (None, w):
        out, out_all = _buffer(gen, T, d, more, at, t, 9.0)
        if weights is None:
            m.moe_permute_backward(y, pos, out)
        else:
            m.moe_unpermute(y, pos, out, topk_w=w)
        ref, size = OR.unpermute(_np(y), held, None if weights is None else _np(w))
        # k additions of products: (k + 1) U of their magnitudes; one rounding of half a step (of fp16's
        # smallest, 2^-24, below its normal range)
        tol = half * np.abs(ref) + 1.01 * (k + 1) * U * size + (2.0 ** -25 if dtype == "f16" else 0)
        assert np.all(np.abs(_np(out) - ref) <= tol)
        inside = torch.zeros_like(out_all, dtype=torch.bool)
        inside[at:at + T * (d + more)].view(-1, d + more)[:, :d] = True
        assert bool((out_all[~inside] == 9).all())
        g, _ = _buffer(gen, T, d, more, at, t)
        d_rows, _ = _buffer(gen, R + spare, d, 0, 0, t, 9.0)
        d_w = torch.full((T, k), 9.0, device="cuda")
        m.moe_unpermute_backward(pos, g, y, weights, d_rows, d_w)
        ref_rows, ref_w, size = OR.unpermute_backward(_np(y), held, None if weights is None else _np(w), _np(g), _np(torch.full_like(d_rows, 9.0)))
        tol = (half + 2 * U) * np.abs(ref_rows) + (2.0 ** -25 if dtype == "f16" else 0)
        assert np.all(np.abs(_np(d_rows) - ref_rows) <= tol)
        assert np.all(np.abs(_np(d_w) - ref_w) <= (d + 2) * U * size)
        one, other = torch.full_like(d_rows, 9.0), torch.full_like(d_w, 9.0)
        m.moe_unpermute_backward(pos, g, None, weights, one, None)
        m.moe_unpermute_backward(pos, g, y, weights, None, other)
        assert torch.equal(one, d_rows) and torch.equal(other, d_w)


def test_no_tokens_and_no_rows():
    m = _m()
    pos = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    x, none = torch.randn(3, 5, device="cuda"), torch.empty(0, 5, device="cuda")
    m.moe_permute(x, pos, none)
    out, d_w = torch.full_like(x, 9.0), torch.full((3, 2), 9.0, device="cuda")
    m.moe_unpermute(none, pos, out)
    m.moe_unpermute_backward(pos, x, none, None, none, d_w)
    assert bool((out == 0).all()) and bool((d_w == 0).all())
    rows = torch.full((4, 5), 9.0, device="cuda")
    m.moe_permute(none, pos[:0], rows)
    m.moe_permute_backward(rows, pos[:0], none)
    m.moe_unpermute_backward(pos[:0], none, rows, None, rows, d_w[:0])
    assert bool((rows == 9).all())


def test_one_gradient_alone_without_tokens_or_rows():
    """An empty gradient is given, though its address is 0."""
    m = _m()
    pos = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    g, w, rows = torch.randn(3, 5, device="cuda"), torch.randn(3, 2, device="cuda"), torch.full((4, 5), 9.0, device="cuda")
    none, no_w = torch.empty(0, 5, device="cuda"), torch.empty(0, 2, device="cuda")
    for weights in (None, w):
        m.moe_unpermute_backward(pos, g, topk_w=weights, d_rows=none)               # no expert of the rank got a row
        m.moe_unpermute_backward(pos, g, none, weights, none)
        d_w = torch.full((3, 2), 9.0, device="cuda")
        m.moe_unpermute_backward(pos, g, none, weights, d_topk_w=d_w)
        assert bool((d_w == 0).all())
        no = None if weights is None else no_w
        m.moe_unpermute_backward(pos[:0], none, rows, no, d_topk_w=no_w)            # no tokens
        m.moe_unpermute_backward(pos[:0], none, topk_w=no, d_rows=rows)
        m.moe_unpermute_backward(pos[:0], none, none, no, none, no_w)               # neither
        m.moe_unpermute_backward(pos[:0], none, none, no, d_topk_w=no_w)
        m.moe_unpermute_backward(pos[:0], none, topk_w=no, d_rows=none)
    assert bool((rows == 9).all())


def test_offsets_beyond_32_bits():
    """Rows 4 MB apart, so that the last ones lie 4.6 GB behind the first."""
    m = _m()
    pitch, R = 1 << 21, 1100
    rows = torch.empty(R * pitch, dtype=torch.bfloat16, device="cuda").view(R, pitch)[:, :24]
    rows.zero_()
    pos = torch.tensor([[R - 1, 0], [1050, 1]], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 24, device="cuda").to(torch.bfloat16)
    m.moe_permute(x, pos, rows)
    assert torch.equal(rows[R - 1], x[0]) and torch.equal(rows[0], x[0]) and torch.equal(rows[1050], x[1])
    assert int((rows != 0).any(1).sum()) == 4
    out = torch.empty_like(x)
    m.moe_unpermute(rows, pos, out)
    assert torch.equal(out, (2 * x.float()).to(torch.bfloat16))
    d_w = torch.empty(2, 2, device="cuda")
    m.moe_unpermute_backward(pos, x, rows, None, None, d_w)
    assert torch.allclose(d_w, x.float().square().sum(1, keepdim=True).expand(2, 2), rtol=1e-5)


def test_captured_on_streams_and_at_once():
    """Sort, rows and sum in a graph replayed over new inputs; two batches on two streams: the bits of the eager calls."""
    m = _m()

    class Batch:
        def __init__(self, seed, T=3000, k=4, E=32, d=520):
            g = torch.Generator(device="cuda").manual_seed(seed)
            self.g, self.T, self.k, self.E = g, T, k, E
            self.ids = torch.randint(0, E + 2, (T, k), generator=g, device="cuda").to(torch.int32)
            self.x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
            self.w = torch.rand(T, k, generator=g, device="cuda")
            e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
            self.pos, self.offsets, self.src = e(T, k, dt=torch.int32), e(E + 1, dt=torch.int32), e(T * k, dt=torch.int32)
            self.rows, self.out, self.d_rows, self.d_w, self.dx = e(T * k, d), e(T, d), e(T * k, d), e(T, k, dt=torch.float32), e(T, d)

        def run(self, stream=None):
            m.moe_sort(self.ids, self.pos, self.offsets, src=self.src, stream=stream)
            m.moe_permute(self.x, self.pos, self.rows, stream=stream)
            m.moe_unpermute(self.rows, self.pos, self.out, topk_w=self.w, stream=stream)
            m.moe_unpermute_backward(self.pos, self.x, self.rows, self.w, self.d_rows, self.d_w, stream=stream)
            m.moe_permute_backward(self.d_rows, self.pos, self.dx, stream=stream)

        def results(self):
            R = int(self.offsets[self.E])
            return [t.clone() for t in (self.pos, self.offsets, self.src[:R], self.rows[:R], self.out, self.d_rows[:R], self.d_w, self.dx)]

    b = Batch(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for r in range(4):
        b.ids.copy_(torch.randint(0, b.E + 2, (b.T, b.k), generator=b.g, device="cuda"))
        b.x.copy_(torch.randn(b.x.shape, generator=b.g, device="cuda"))
        b.run()
        torch.cuda.synchronize()
        want = b.results()
        for t in (b.pos, b.offsets, b.out, b.d_w, b.dx):
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, b.results())), r
    pair = [Batch(2), Batch(3, T=5000)]
    want = []
    for p in pair:
        p.run()
        torch.cuda.synchronize()
        want.append(p.results())
    streams = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    for i in range(4):
        for p, s in zip(pair, streams):
            if i % 2:
                p.run(stream=s if i == 1 else s.cuda_stream)     # given as an argument, an object or a raw handle
            else:
                with torch.cuda.stream(s):
                    p.run()
    torch.cuda.synchronize()
    for p, ref in zip(pair, want):
        assert all(torch.equal(u, v) for u, v in zip(ref, p.results()))


def test_gradients_are_differences():
    """The loss <g, sum back of rows and weights> along random directions, in fp32."""
    m = _m()
    gen = torch.Generator(device="cuda").manual_seed(0)
    rng = np.random.default_rng(0)
    T, k, d = 9, 3, 50
    ids = rng.integers(0, 5, (T, k)).astype(np.int32)
    pos, _, offsets = _sorted(ids, 4)
    R, held = int(offsets[4]), _np(pos).astype(np.int64)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    y, w, g = rn(R, d), rn(T, k), rn(T, d)
    d_rows, d_w, dx = torch.zeros_like(y), torch.zeros_like(w), torch.zeros_like(g)
    m.moe_unpermute_backward(pos, g, y, w, d_rows, d_w)
    m.moe_permute_backward(y, pos, dx)
    for _ in range(3):
        vy, vw = rng.standard_normal(y.shape), rng.standard_normal(w.shape)
        f = [(_np(g) * OR.unpermute(_np(y) + s * vy, held, _np(w) + s * vw)[0]).sum() for s in (1e-4, -1e-4)]
        assert np.isclose((f[0] - f[1]) / 2e-4, (_np(d_rows) * vy).sum() + (_np(d_w) * vw).sum(), rtol=1e-4, atol=1e-4)
        vx = rng.standard_normal(g.shape)
        moved = OR.permute(vx, held, np.zeros(y.shape))
        assert np.isclose((_np(dx) * vx).sum(), (moved * _np(y)).sum(), rtol=1e-4, atol=1e-4)
