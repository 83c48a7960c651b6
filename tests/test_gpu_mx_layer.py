"""The sorted rows and the 4-bit products run together as a layer uses them:
router product, routing, sort, tokens to rows, gated up and down products with
4-bit weights (rows in 16 bits, or quantised), weighted sum back; and the training
step around them, with each expert's dense products and all gradients.  Also
captured into a graph, on two streams at once, on another stream, and over
buffers larger than 4 GB."""
import numpy as np
import pytest
import torch

from oracle import linear as OL
from oracle import mx as OM
from oracle import route as OR
from oracle import rows as OS

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16


def _m():
    import moe_expert_tile_amd as m
    return m


def _np(t):
    return t.detach().double().cpu().numpy()


def _e(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


class _Serving:
    """A rank's layer with 4-bit experts `first` .. `first` + E - 1 of `total`."""

    def __init__(self, T=70, total=16, E=8, first=4, k=4, d=256, f=192, seed=0, packed=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.T, self.E, self.first, self.k, self.d, self.f, self.packed = gen, T, E, first, k, d, f, packed
        self.x = self.randn(T, d)
        self.w_router = self.randn(total, d, std=d ** -0.5)
        up, down = self.randn(E * 2 * f, d, std=0.08), self.randn(E * d, f, std=0.08)
        self.up, self.up_scale = _e(E, 2 * f, d // 2, dtype=torch.uint8), _e(E, 2 * f, d // 32, dtype=torch.uint8)
        self.down, self.down_scale = _e(E, d, f // 2, dtype=torch.uint8), _e(E, d, f // 32, dtype=torch.uint8)
        _m().moe_mx_quantize(up, self.up.view(-1, d // 2), self.up_scale.view(-1, d // 32))
        _m().moe_mx_quantize(down, self.down.view(-1, f // 2), self.down_scale.view(-1, f // 32))
        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        self.logits, self.ids, self.w = _e(T, total, dtype=f32), _e(T, k, dtype=i32), _e(T, k, dtype=f32)
        self.pos, self.offsets = _e(T, k, dtype=i32), _e(E + 1, dtype=i32)
        self.rows, self.h, self.y, self.out = _e(T * k, d), _e(T * k, f), _e(T * k, d), _e(T, d)
        self.xq, self.xs = _e(T * k, d // 2, dtype=u8), _e(T * k, d // 32, dtype=u8)
        self.hq, self.hs = _e(T * k, f // 2, dtype=u8), _e(T * k, f // 32, dtype=u8)

    def randn(self, *s, std=1.0):
        return (torch.randn(*s, generator=self.gen, device="cuda") * std).to(BF)

    def run(self, stream=None):
        m = _m()
        s = dict(stream=stream)
        m.moe_linear(self.x, self.w_router, self.logits, **s)
        m.moe_route(self.logits, self.ids, self.w, renorm=True, **s)
        m.moe_sort(self.ids, self.pos, self.offsets, first=self.first, **s)
        m.moe_permute(self.x, self.pos, self.rows, **s)
        if self.packed:
            m.moe_mx_quantize(self.rows, self.xq, self.xs, **s)
            m.moe_mx_linear(self.xq, self.up, self.up_scale, self.h, offsets=self.offsets, x_scale=self.xs, act=m.ACT_SWIGLU, **s)
            m.moe_mx_quantize(self.h, self.hq, self.hs, **s)
            m.moe_mx_linear(self.hq, self.down, self.down_scale, self.y, offsets=self.offsets, x_scale=self.hs, **s)
        else:
            m.moe_mx_linear(self.rows, self.up, self.up_scale, self.h, offsets=self.offsets, act=m.ACT_SWIGLU, **s)
            m.moe_mx_linear(self.h, self.down, self.down_scale, self.y, offsets=self.offsets, **s)
        m.moe_unpermute(self.y, self.pos, self.out, topk_w=self.w, **s)

    def results(self):
        R = int(self.offsets[self.E])
        return [t.clone() for t in (self.logits, self.ids, self.w, self.pos, self.offsets, self.rows[:R], self.h[:R], self.y[:R], self.out)]


@pytest.mark.parametrize("packed", [False, True])
def test_serving_layer(packed):
    """Each step against its definition in 64 bits on the step before's results."""
    L = _Serving(packed=packed)
    L.run()
    logits = _np(L.logits)
    S = np.abs(_np(L.x)) @ np.abs(_np(L.w_router)).T
    assert np.all(np.abs(logits - _np(L.x) @ _np(L.w_router).T) <= (L.d + 2) * U * S)
    ids, w = OR.route(logits, L.k, renorm=True)
    assert np.array_equal(ids, L.ids.cpu().numpy()) and np.allclose(_np(L.w), w, rtol=2.0 ** -18)
    pos, src, offsets = OS.sort(ids, L.E, L.first)
    R = offsets[-1]
    assert np.array_equal(pos, L.pos.cpu().numpy()) and np.array_equal(offsets, L.offsets.cpu().numpy()) and 0 < R < L.T * L.k
    assert np.array_equal(_np(L.rows[:R]), _np(L.x)[src // L.k])
    up, down = OM.values(L.up.cpu().numpy(), L.up_scale.cpu().numpy()), OM.values(L.down.cpu().numpy(), L.down_scale.cpu().numpy())
    x, h = _np(L.rows), _np(L.h)
    if packed:
        assert all(np.array_equal(a.cpu().numpy()[:R], b) for t, q, s in ((L.rows, L.xq, L.xs), (L.h, L.hq, L.hs))
                   for a, b in zip((q, s), OM.quantize(_np(t[:R]))))
        x, h = (OM.values(q.cpu().numpy(), s.cpu().numpy()) for q, s in ((L.xq, L.xs), (L.hq, L.hs)))
    half = 2.0 ** -8
    from test_gpu_linear import _forward_error
    for a, wt, act, got in ((x, up, "swiglu", L.h), (h, down, "none", L.y)):
        for e in range(L.E):
            lo, hi = offsets[e], offsets[e + 1]
            if hi == lo:
                continue
            z = OL.product(a[lo:hi], wt[e])
            _, ey = _forward_error(a[lo:hi], wt[e], None, act, z)
            y = OL.apply(act, z)
            assert np.all(np.abs(_np(got[lo:hi]) - y) <= ey * (1 + half) + half * np.abs(y))
    ref, size = OS.unpermute(_np(L.y[:R]), pos, _np(L.w))
    assert np.all(np.abs(_np(L.out) - ref) <= half * np.abs(ref) + 1.01 * (L.k + 1) * U * size)
    assert np.abs(ref).max() > 0.1


@pytest.mark.parametrize("packed", [False, True])
def test_captured_and_replayed(packed):
    L = _Serving(T=300, seed=3, packed=packed)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run()
    for r in range(4):
        L.x.copy_(L.randn(*L.x.shape))
        L.run()
        torch.cuda.synchronize()
        want = L.results()
        for t in (L.logits, L.w, L.out, L.h, L.y, L.rows):
            t.fill_(5.0)
        L.offsets.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, L.results())), r


def test_two_layers_at_once_and_given_streams():
    layers = [_Serving(T=400, seed=1), _Serving(T=900, seed=2, packed=True)]
    want = []
    for L in layers:
        L.run()
        torch.cuda.synchronize()
        want.append(L.results())
    streams = [torch.cuda.Stream() for _ in layers]
    for how in ("current", "object", "handle", "current"):
        torch.cuda.synchronize()
        for L, s in zip(layers, streams):
            if how == "current":
                with torch.cuda.stream(s):
                    L.run()
            else:
                L.run(stream=s if how == "object" else s.cuda_stream)
        torch.cuda.synchronize()
        for L, ref in zip(layers, want):
            assert all(torch.equal(a, b) for a, b in zip(ref, L.results())), how


@pytest.mark.parametrize("M,N,K,E", [(5, 300, 2048, 3), (900, 200, 544, 4), (4000, 520, 288, 2)])
def test_the_same_call_gives_the_same_bits(M, N, K, E):
    m = _m()
    gen = torch.Generator(device="cuda").manual_seed(M)
    w = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.randint(118, 122, (E, N, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    off = torch.linspace(0, M, E + 1, device="cuda").to(torch.int32)
    x = torch.randn(M, K, generator=gen, device="cuda").to(BF)
    xq, xs = _e(M, K // 2, dtype=torch.uint8), _e(M, K // 32, dtype=torch.uint8)
    m.moe_mx_quantize(x, xq, xs)
    runs = []
    for _ in range(4):
        a, b = _e(M, N), _e(M, N)
        m.moe_mx_linear(x, w, s, a, offsets=off)
        m.moe_mx_linear(xq, w, s, b, offsets=off, x_scale=xs)
        runs.append((a, b))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for r in runs[1:] for p, q in zip(runs[0], r))


def test_training_step_around_the_sorted_rows():
    """Sort, rows, each expert's dense products and the weighted sum, and back: the
    gradients of <g, out> for the experts' weights, the tokens and the logits, along
    random directions against differences in float64."""
    m = _m()
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, E, k, d, f = 40, 6, 2, 64, 48

    def randn(*s, std=1.0):
        return (torch.randn(*s, generator=gen, device="cuda") * std).to(torch.float16)

    x, up, down, g = randn(T, d), randn(E, 2 * f, d, std=0.15), randn(E, d, f, std=0.15), randn(T, d)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    ids, w = _e(T, k, dtype=i32), _e(T, k, dtype=f32)
    m.moe_route(logits, ids, w, renorm=True)
    pos, offsets = _e(T, k, dtype=i32), _e(E + 1, dtype=i32)
    m.moe_sort(ids, pos, offsets)
    R = T * k
    rows, h, pre, y, out = (_e(*s, dtype=f16) for s in ((R, d), (R, f), (R, 2 * f), (R, d), (T, d)))
    m.moe_permute(x, pos, rows)
    off = offsets.tolist()
    pieces = [(e, slice(off[e], off[e + 1])) for e in range(E) if off[e + 1] > off[e]]
    for e, r in pieces:
        m.moe_linear(rows[r], up[e], h[r], pre=pre[r], act=m.ACT_SWIGLU)
        m.moe_linear(h[r], down[e], y[r])
    m.moe_unpermute(y, pos, out, topk_w=w)
    d_y, d_w, d_h, d_rows, dx = _e(R, d, dtype=f16), _e(T, k, dtype=f32), _e(R, f, dtype=f16), _e(R, d, dtype=f16), _e(T, d, dtype=f16)
    d_up, d_down, d_logits = torch.zeros_like(up), torch.zeros_like(down), torch.zeros_like(logits)
    m.moe_unpermute_backward(pos, g, y, w, d_y, d_w)
    for e, r in pieces:
        m.moe_linear_backward(h[r], down[e], d_y[r], dx=d_h[r], dw=d_down[e])
        m.moe_linear_backward(rows[r], up[e], d_h[r], dx=d_rows[r], dw=d_up[e], pre=pre[r], act=m.ACT_SWIGLU)
    m.moe_permute_backward(d_rows, pos, dx)
    m.moe_route_backward(logits, ids, w, d_w, d_logits, renorm=True)
    torch.cuda.synchronize()
    held, idn, gn = np.ones((T, k), bool), ids.cpu().numpy(), _np(g)

    def loss(x, up, down, logits):
        wt = OR.weights_of(logits, idn, held, "softmax", True, 1.0)
        total = 0.0
        for t in range(T):
            for j in range(k):
                e = idn[t, j]
                total += wt[t, j] * gn[t] @ (down[e] @ OL.apply("swiglu", (up[e] @ x[t])[None])[0])
        return total

    at = [_np(v) for v in (x, up, down, logits)]
    grads = [_np(v) for v in (dx, d_up, d_down, d_logits)]
    rng = np.random.default_rng(0)
    for i in range(4):
        for _ in range(2):
            v = rng.standard_normal(at[i].shape)
            moved = [[a + s * 1e-5 * v if n == i else a for n, a in enumerate(at)] for s in (1, -1)]
            quotient = (loss(*moved[0]) - loss(*moved[1])) / 2e-5
            # fp16 roundings of h, pre, y and of the gradients passed on: each half a step, 2^-11 of its
            # value, at most eight in a chain; an entry's error enters with the direction's size
            size = np.abs(grads[i] * v).sum()
            assert abs((grads[i] * v).sum() - quotient) <= 8 * 2.0 ** -11 * size + 1e-6 * abs(quotient), i


def test_buffers_beyond_32_bits():
    """Rows and weights that lie more than 4 GB behind the first."""
    m = _m()
    K, N = 64, 32
    pitch = 1 << 21                                      # bytes between packed rows
    R = 2200
    xq = torch.empty(R * pitch, dtype=torch.uint8, device="cuda").view(R, pitch)[:, :K // 2]
    gen = torch.Generator(device="cuda").manual_seed(0)
    small = torch.randint(0, 256, (R, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    xq.copy_(small)
    xs = torch.full((R, K // 32), 127, dtype=torch.uint8, device="cuda")
    gap = 5 << 30                                        # bytes between two experts' weights
    whole = torch.empty(gap + N * K // 2, dtype=torch.uint8, device="cuda")
    w = whole.as_strided((2, N, K // 2), (gap, K // 2, 1))
    w.copy_(torch.randint(0, 256, (2, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8))
    s = torch.full((2, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 7, R], dtype=torch.int32, device="cuda")
    wide = torch.empty(R * (pitch // 4), dtype=torch.float32, device="cuda").view(R, pitch // 4)[:, :N]
    out = torch.empty(R, N, device="cuda")
    m.moe_mx_linear(xq, w, s, wide, offsets=off, x_scale=xs)
    m.moe_mx_linear(small, w.contiguous(), s, out, offsets=off, x_scale=xs)
    assert torch.equal(wide, out) and float(out.abs().max()) > 0
    x16 = torch.empty(R, K, dtype=BF, device="cuda")
    m.moe_mx_dequantize(xq, xs, x16)
    far = torch.empty(R * (pitch // 2), dtype=BF, device="cuda").view(R, pitch // 2)[:, :K]
    far.copy_(x16)
    m.moe_mx_linear(far, w, s, wide, offsets=off)
    m.moe_mx_linear(x16, w.contiguous(), s, out, offsets=off)
    assert torch.equal(wide, out)
