"""The scale step's gradient, and the operators around the experts run
together as a layer uses them: router product, routing, plan, expert FFN and
combine, scale, shared expert; then the gradients back to the router's
weights.  Also under HIP graph capture, on another stream, and in the order of
two calls that share nothing.
"""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import say
from oracle import linear as OL
from oracle import plan as OP
from oracle import route as OR

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _m():
    import moe_expert_tile_amd as m
    return m


def _np(t):
    return t.detach().double().cpu().numpy()


def _share(T, E, k, d, f=128, seed=0, tokens=None, rank=0, W=1):
    """A planned rank share over random routing, its ids and positions."""
    m = _m()
    tokens = tokens or [T]
    rng = np.random.default_rng(seed)
    N = sum(tokens)
    ids = np.argsort(rng.random((N, E)), axis=1)[:, :k].astype(np.int32)
    E_l = E // W
    pl = OP.build_plan(ids, tuple(tokens), rank, E_l, 32, 1)
    sh = m.RankShare(m.Shape(W, rank, E_l, k, d, f, 32, tokens, pl.R))
    ids_d = torch.from_numpy(ids).cuda()
    sh.plan(ids_d, torch.zeros(max(1, pl.R), d, dtype=torch.bfloat16, device="cuda"), materialize=False)
    return sh, ids_d, torch.from_numpy(np.ascontiguousarray(pl.pos)).long().cuda()


@pytest.mark.parametrize("tokens,rank,E,k,d", [([1], 0, 4, 1, 256), ([7], 0, 8, 8, 512), ([65], 0, 32, 6, 2048),
                                               ([40, 0, 33], 2, 9, 2, 1280), ([0, 5], 0, 4, 2, 256),
                                               ([300], 0, 64, 32, 256), ([33], 0, 16, 3, 7168), ([9], 0, 8, 2, 65536),
                                               ([2000], 0, 32, 4, 768)])
def test_scale_backward(tokens, rank, E, k, d):
    say(f"[scale back] tokens={tokens} rank={rank} E={E} k={k} d={d}")
    sh, _, pos = _share(0, E, k, d, tokens=tokens, rank=rank, W=len(tokens))
    T = tokens[rank]
    gen = torch.Generator(device="cuda").manual_seed(d + k)
    rows = max(1, T * k)
    sh.recv[rank] = torch.randn(rows, d, generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.rand(max(1, T), k, generator=gen, device="cuda")
    w[0, 0] = 0
    g = torch.randn(max(1, T), d, generator=gen, device="cuda").to(torch.bfloat16)
    d_recv, d_w = torch.full_like(sh.recv[rank], 9.0), torch.full_like(w, 9.0)
    sh.scale_backward(w, g, d_recv, d_w)
    assert sh.status() == 0
    if T == 0:
        assert bool((d_recv == 9).all()) and bool((d_w == 9).all())
        return
    ref = w.double().unsqueeze(2) * g.double().unsqueeze(1)                   # [T, k, d]
    got = d_recv[pos.view(-1)].view(T, k, d).double()
    # one rounding to 24 bits, one to bf16 (half a step 2^-8 with its eps of 2^-7)
    assert bool(((got - ref).abs() <= (2.0 ** -8 + 2 * U) * ref.abs()).all())
    prod = sh.recv[rank][pos.view(-1)].view(T, k, d).double() * g.double().unsqueeze(1)
    assert bool(((d_w.double() - prod.sum(2)).abs() <= (d + 2) * U * prod.abs().sum(2)).all())
    # one of the two alone: the same bits
    a, b = torch.full_like(d_recv, 9.0), torch.full_like(d_w, 9.0)
    sh.scale_backward(w, g, a, None)
    sh.scale_backward(w, g, None, b)
    assert torch.equal(a, d_recv) and torch.equal(b, d_w)
    # what a gradient does not need may be missing
    m = _m()
    b.fill_(9.0)
    m.moe_scale_backward(sh.shape, sh.plan_ws, sh.recv[rank], None, g, None, b)
    m.moe_scale_backward(sh.shape, sh.plan_ws, None, w, g, a.fill_(9.0), None)
    assert torch.equal(a, d_recv) and torch.equal(b, d_w)


def test_scale_backward_after_a_routing_error_does_nothing():
    m = _m()
    sh, ids, _ = _share(16, 8, 2, 256)
    ids[3, 1] = 99
    sh.plan(ids, torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda"), materialize=False)
    a, b = torch.full((32, 256), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((16, 2), 9.0, device="cuda")
    sh.scale_backward(torch.ones(16, 2, device="cuda"), torch.ones(16, 256, dtype=torch.bfloat16, device="cuda"), a, b)
    assert sh.status() == m.MOE_EROUTING
    assert bool((a == 9).all()) and bool((b == 9).all())


class _Layer:
    """One rank's layer with its own router and shared expert (W = 1)."""

    def __init__(self, T=96, E=16, k=4, d=512, f=256, seed=0):
        m = _m()
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*s, std=1.0):
            return (torch.randn(*s, generator=gen, device="cuda") * std).to(torch.bfloat16)

        self.T, self.E, self.k, self.d, self.f = T, E, k, d, f
        self.x = randn(T, d)
        self.w_router = randn(E, d, std=d ** -0.5)
        self.bias = torch.randn(E, generator=gen, device="cuda") * 0.1
        self.w_gate_up, self.w_down = randn(E, 2 * f, d, std=0.05), randn(E, d, f, std=0.05)
        self.ws_up, self.ws_down = randn(2 * f, d, std=0.05), randn(d, f, std=0.05)
        self.g = randn(T, d)
        self.share = m.RankShare(m.Shape(1, 0, E, k, d, f, 32, [T], T * k))
        e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        self.logits, self.ids, self.w = e(T, E, dt=torch.float32), e(T, k, dt=torch.int32), e(T, k, dt=torch.float32)
        self.hs, self.out = e(T, f), e(T, d)
        self.x_recv = e(T * k, d)
        self.d_recv, self.d_w = e(T * k, d), e(T, k, dt=torch.float32)
        self.d_logits, self.d_router, self.dx = e(T, E, dt=torch.float32), e(E, d), e(T, d)
        self.opts = dict(score=m.SCORE_SIGMOID, renorm=True, scale=2.5)

    def route(self):
        m = _m()
        m.moe_linear(self.x, self.w_router, self.logits)
        m.moe_route(self.logits, self.ids, self.w, bias=self.bias, n_group=4, topk_group=2, group_score=m.GROUP_TOP2,
                    **self.opts)

    def experts(self):
        # dispatch: every (token, slot) of the one rank, in order
        self.x_recv.copy_(self.x.repeat_interleave(self.k, 0))
        self.share.plan(self.ids, self.x_recv)
        self.share.combine(self.w_gate_up, self.w_down, mode=_m().MODE_SERIAL)

    def finish(self):
        m = _m()
        self.share.scale(self.w)
        m.moe_linear(self.x, self.ws_up, self.hs, act=m.ACT_SWIGLU)
        m.moe_linear(self.hs, self.ws_down, self.out, residual=self.share.out)

    def backward(self):
        m = _m()
        self.share.scale_backward(self.w, self.g, self.d_recv, self.d_w)
        m.moe_route_backward(self.logits, self.ids, self.w, self.d_w, self.d_logits, **self.opts)
        m.moe_linear_backward(self.x, self.w_router, self.d_logits, dx=self.dx, dw=self.d_router)

    def results(self):
        return [t.clone() for t in (self.logits, self.ids, self.w, self.out, self.d_recv, self.d_w, self.d_logits,
                                    self.d_router, self.dx)]


def test_layer_forward_and_gradient():
    m = _m()
    L = _Layer()
    L.route()
    L.experts()
    L.finish()
    L.backward()
    assert L.share.status() == m.MOE_OK
    logits = _np(L.logits)
    x, wr = _np(L.x), _np(L.w_router)
    S = np.abs(x) @ np.abs(wr).T
    assert np.all(np.abs(logits - x @ wr.T) <= (L.d + 2) * U * S)
    ids, w = OR.route(logits, L.k, kind="sigmoid", bias=_np(L.bias), renorm=True, n_group=4, topk_group=2, top2=True,
                      scale=2.5)
    assert np.array_equal(ids, L.ids.cpu().numpy()) and np.allclose(_np(L.w), w, rtol=2.0 ** -18)
    # the layer's output, token by token in float64 from the definition (the experts' h and y rounded to bf16)
    wgu, wd = _np(L.w_gate_up), _np(L.w_down)
    out = OL.apply("swiglu", x @ _np(L.ws_up).T) @ _np(L.ws_down).T
    y = np.zeros((L.T, L.k, L.d))
    for t in range(L.T):
        for j in range(L.k):
            e = ids[t, j]
            y[t, j] = wd[e] @ OL.apply("swiglu", (wgu[e] @ x[t])[None])[0]
    routed = (w[:, :, None] * y).sum(1)
    err = np.abs(_np(L.out) - (out + routed))
    # the path's stated tolerance for bf16 outputs
    assert np.all(err <= 2e-2 + 1e-2 * np.abs(out + routed)), err.max()
    # gradient of <g, layer output> through the gate weights, with the rows that came back as constants
    pl = OP.build_plan(ids, (L.T,), 0, L.E, 32, 1)
    rows = _np(L.share.recv[0])[pl.pos]
    g = _np(L.g)
    d_w = (rows * g[:, None, :]).sum(2)
    assert np.all(np.abs(_np(L.d_w) - d_w) <= (L.d + 2) * U * np.abs(rows * g[:, None, :]).sum(2))
    held = np.ones_like(ids, bool)
    d_logits = OR.route_backward(logits, ids, held, d_w, kind="sigmoid", renorm=True, scale=2.5)
    tol = 2.0 ** -17 * 2.5 * np.abs(d_w).max() + (L.d + 2) * U * np.abs(rows * g[:, None, :]).sum(2).max() * 2.5
    assert np.all(np.abs(_np(L.d_logits) - d_logits) <= tol)
    half = 2.0 ** -8
    for got, ref, mag in ((_np(L.d_router), d_logits.T @ x, np.abs(d_logits).T @ np.abs(x)),
                          (_np(L.dx), d_logits @ wr, np.abs(d_logits) @ np.abs(wr))):
        slack = tol * (np.abs(x).sum(0)[None] if got.shape[0] == L.E else np.abs(wr).sum(0)[None])
        assert np.all(np.abs(got - ref) <= half * (mag + np.abs(ref)) * 1.01 + slack * 1.01)
    # ... and against differences: the loss along random directions of the router's weights
    rng = np.random.default_rng(0)
    for _ in range(4):
        v = rng.standard_normal(wr.shape)
        h = 1e-5
        f = [(g * (OR.weights_of(x @ (wr + s * h * v).T, ids, held, "sigmoid", True, 2.5)[:, :, None] * rows).sum(1)).sum()
             for s in (1, -1)]
        quotient = (f[0] - f[1]) / (2 * h)
        # every entry of the gradient is off by at most the bound above
        bound = (np.abs(v) * (half * 2 * (np.abs(d_logits).T @ np.abs(x)) * 1.01 + tol * np.abs(x).sum(0)[None] * 1.01)).sum()
        assert abs((v * _np(L.d_router)).sum() - quotient) <= bound + 1e-5 * abs(quotient)


def test_captured_and_replayed():
    """Router, routing, plan, scale, shared expert and the gradients in one HIP
    graph; new inputs between replays, each replay against the eager calls."""
    L = _Layer(T=130, seed=3)
    L.route()
    L.experts()
    L.finish()
    L.backward()
    torch.cuda.synchronize()

    def steps():
        L.route()
        L.share.plan(L.ids, L.x_recv, materialize=False)
        L.finish()
        L.backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for r in range(4):
        gen = torch.Generator(device="cuda").manual_seed(50 + r)
        L.x.copy_(torch.randn(L.x.shape, generator=gen, device="cuda"))
        steps()
        torch.cuda.synchronize()
        want = L.results()
        for t in (L.logits, L.w, L.out, L.d_recv, L.d_w, L.d_logits, L.d_router, L.dx):
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, L.results()):
            assert torch.equal(a, b), r


def test_calls_on_two_streams_at_once():
    """Two layers on two streams, workspaces from the allocator: the same bits as one after the other."""
    layers = [_Layer(T=300, seed=s) for s in (1, 2)]
    want = []
    for L in layers:
        L.route()
        L.experts()
        L.finish()
        L.backward()
        torch.cuda.synchronize()
        want.append(L.results())
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(3):
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.route()
                L.finish()
                L.backward()
    torch.cuda.synchronize()
    for L, ref in zip(layers, want):
        for a, b in zip(ref, L.results()):
            assert torch.equal(a, b)


def test_given_streams():
    """A stream given as an argument, as an object and as a raw handle."""
    m = _m()
    s = torch.cuda.Stream()
    x = torch.randn(256, 512, device="cuda").to(torch.bfloat16)
    w = torch.randn(96, 512, device="cuda").to(torch.bfloat16)
    g = torch.randn(256, 96, device="cuda").to(torch.bfloat16)
    ref, dw = torch.empty(256, 96, device="cuda"), torch.empty_like(w)
    m.moe_linear(x, w, ref)
    m.moe_linear_backward(x, w, g, dw=dw)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        out, got = torch.zeros_like(ref), torch.zeros_like(dw)
        torch.cuda.synchronize()
        m.moe_linear(x, w, out, stream=stream)
        m.moe_linear_backward(x, w, g, dw=got, stream=stream)
        ids, wt = torch.zeros(256, 4, dtype=torch.int32, device="cuda"), torch.zeros(256, 4, device="cuda")
        m.moe_route(out, ids, wt, stream=stream)
        s.synchronize()
        assert torch.equal(out, ref) and torch.equal(got, dw)
        assert bool((wt > 0).all())


def test_results_do_not_depend_on_timing():
    """The same call twice gives the same bits: sums split over workgroups are joined in a fixed order."""
    m = _m()
    x = torch.randn(2000, 2048, device="cuda").to(torch.bfloat16)
    w = torch.randn(60, 2048, device="cuda").to(torch.bfloat16)
    g = torch.randn(2000, 60, device="cuda")
    runs = []
    for _ in range(4):
        out, dx, dw = torch.empty(2000, 60, device="cuda"), torch.empty_like(x), torch.empty_like(w)
        db = torch.empty(60, dtype=torch.bfloat16, device="cuda")
        m.moe_linear(x, w, out)
        m.moe_linear_backward(x, w, g, dx=dx, dw=dw, dbias=db)
        runs.append((out, dx, dw, db))
    torch.cuda.synchronize()
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_router_of_the_named_workloads():
    """The repository's workloads: their expert counts and top-k with the
    binding's routing in front of their plan."""
    m = _m()
    for name in ("tiny", "decode_tb32"):
        cfg = synth.get_config(name)
        x = torch.from_numpy(synth.activations(cfg).view(np.int16)).view(torch.bfloat16).cuda()
        gen = torch.Generator(device="cuda").manual_seed(7)
        wr = (torch.randn(cfg.E, cfg.d, generator=gen, device="cuda") * cfg.d ** -0.5).to(torch.bfloat16)
        logits = torch.empty(cfg.N, cfg.E, device="cuda")
        ids, w = torch.empty(cfg.N, cfg.k, dtype=torch.int32, device="cuda"), torch.empty(cfg.N, cfg.k, device="cuda")
        m.moe_linear(x, wr, logits)
        m.moe_route(logits, ids, w, renorm=cfg.weights == "renorm")
        host = ids.cpu().numpy()
        pl = OP.build_plan(host, cfg.tokens, cfg.rank, cfg.E_l, cfg.tb_m, 1)
        sh = m.RankShare(m.Shape(cfg.W, cfg.rank, cfg.E_l, cfg.k, cfg.d, cfg.f, cfg.tb_m, cfg.tokens, pl.R))
        sh.plan(ids, torch.zeros(max(1, pl.R), cfg.d, dtype=torch.bfloat16, device="cuda"))
        assert sh.status() == m.MOE_OK and sh.header()["M"] == pl.M
