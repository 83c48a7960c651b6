"""The dense product's fp16 gradients at both ends of fp16's range: d loss / d
(x w^T + bias) is rounded to 16 bits inside, its results are not to show more of
that than half a step of each value or 2^-39 of the largest one.

Tolerances are those of test_gpu_linear.py (u = 2^-24; half = 2^-11, half a
step of fp16), with that bound in the place of fp16's own smallest step: the
largest value is brought to 2^14 at least, where fp16's finest absolute error is
2^-25, 2^-39 of it.  The results are fp16 and keep its smallest step, 2^-25.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import linear as OL
from test_gpu_linear import EACH_TILE

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -11
F16, F32 = torch.float16, torch.float32


def _m():
    import moe_expert_tile_amd as m
    return m


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _run(a, act, ws=None):
    m = _m()
    got = {"dx": torch.full_like(a["x"], 9.0), "dw": torch.full_like(a["w"], 9.0),
           "dbias": torch.full((a["w"].shape[0],), 9.0, dtype=F16, device="cuda")}
    m.moe_linear_backward(a["x"], a["w"], a["d_out"], pre=a["pre"], act=getattr(m, "ACT_" + act.upper()), ws=ws, **got)
    torch.cuda.synchronize()
    return got


def _check(a, act, got, sizable=()):
    x, w, g, pre = _np(a["x"]), _np(a["w"]), _np(a["d_out"]), _np(a["pre"])
    n, M = len(w), len(x)
    dz = OL.dz(act, g, pre)
    if act == "none":
        e32 = 0 * np.abs(dz)
    elif act == "swiglu":
        N = g.shape[1]
        z = np.abs(np.concatenate([pre[:, :N]] * 2, 1))
        e32 = (16 + 64 * z) * U * np.concatenate([np.abs(g * pre[:, N:]), np.abs(g * pre[:, :N])], 1)
    else:
        e32 = (16 + 64 * np.abs(pre) * (1 + pre ** 2)) * U * np.abs(g)
    edz = HALF * np.abs(dz) + (1 + HALF) * e32 + 2.0 ** -39 * np.abs(dz).max(initial=0)
    for name, ref, err in (("dx", dz @ w, edz @ np.abs(w) + (n + 8) * U * (np.abs(dz) + edz) @ np.abs(w)),
                           ("dw", dz.T @ x, edz.T @ np.abs(x) + (M + 64) * U * (np.abs(dz) + edz).T @ np.abs(x)),
                           ("dbias", dz.sum(0), (e32 + (M + 2) * U * np.abs(dz)).sum(0))):
        bound = err * (1 + HALF) + HALF * np.abs(ref) + 2.0 ** -25
        held = np.abs(ref) + bound < 65504          # by fp16
        d = np.abs(_np(got[name]) - ref)[held]
        assert np.all(d <= bound[held]), (name, (d - bound[held]).max())
        if name in sizable:     # results well above fp16's smallest step, so that the bound says something
            assert np.abs(ref).max() > 2.0 ** -14, (name, np.abs(ref).max())


def _inputs(M, N, K, act, out, seed, size, xs, ws):
    """Positive x, w and d_out about xs, ws and size."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.rand(*s, generator=gen, device="cuda") + 0.5

    n = 2 * N if act == "swiglu" else N
    pre = torch.randn(M, n, generator=gen, device="cuda").to(F16) if act != "none" else None
    return dict(x=(rand(M, K) * xs).to(F16), w=(rand(n, K) * ws).to(F16), pre=pre, d_out=(rand(M, N) * size).to(out))


# sizes that take several tiles, whole and split, with odd and even n
@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (200, 64, 136), (2000, 61, 520), (700, 1500, 264), (8192, 64, 1032)])
@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
@pytest.mark.parametrize("exp", [-22, -34, 18])
def test_gradients_far_from_one(M, N, K, act, exp):
    """2^-22 is a mean's gradient over four million values; 2^18 lies beyond fp16."""
    size, n = 2.0 ** exp, 2 * N if act == "swiglu" else N
    # operands that bring the sums over M rows and n columns to about 2^4, within fp16's normal numbers
    # (8192 rows of 2^18 times 2^-13 are 2^18: that dw has no fp16 value and is not compared)
    xs, ws = (min(2.0 ** 12, max(2.0 ** -13, 2.0 ** 4 / (size * terms))) for terms in (M, n))
    a = _inputs(M, N, K, act, F32, M + N, size, xs, ws)
    say(f"[linear range] {M}x{N}x{K} {act} 2^{exp}")
    _check(a, act, _run(a, act), () if exp == -34 else ("dx", "dw"))


@pytest.mark.parametrize("d_out,up", [(2.0 ** -10, 2.0 ** -20), (2.0 ** 10, 2.0 ** 10)])
def test_gated_gradients_of_16_bit_inputs(d_out, up):
    """Within fp16 both, their product is not: values of an up projection far from one."""
    size = d_out * up
    M, N, K = 4096, 96, 264
    a = _inputs(M, N, K, "swiglu", F16, 5, d_out, min(2.0 ** 12, 2.0 ** 4 / (size * M)), min(2.0 ** 12, 2.0 ** 4 / (size * 2 * N)))
    a["pre"][:, N:] = (a["pre"][:, N:].float() * up).to(F16)
    a["pre"][:, :N] = -12.0     # silu's value there is near 0, its slope as well: the halves' sizes differ
    a["pre"][:, :N:2] = 2.0
    _check(a, "swiglu", _run(a, "swiglu"), ("dx",))


def test_a_wide_range_within_one_call():
    """Rows from 1 to 2^-30 of the largest: each row of dx to its own accuracy,
    to 2^-39 of the largest value."""
    M, N, K = 300, 128, 136
    a = _inputs(M, N, K, "none", F32, 6, 1.0, 2.0 ** -6, 1.0)
    a["d_out"] *= torch.exp2(-(torch.arange(M, device="cuda") % 31).float()).view(M, 1)
    _check(a, "none", _run(a, "none"), ("dx", "dw"))
    # the largest of all is one value of a single row
    a["d_out"][17, 5] = 2.0 ** 12
    _check(a, "none", _run(a, "none"), ("dx", "dw"))


def test_empty_zero_and_infinite_gradients():
    m = _m()
    a = _inputs(130, 60, 136, "none", F32, 7, 2.0 ** -24, 1.0, 64.0)
    need = m.moe_linear_sizes(m.moe_linear_desc(130, 60, 136, 1, 2, 0, 0))["backward_bytes"]
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")    # NaNs: its contents do not matter
    whole = _run(a, "none", ws)
    _check(a, "none", whole, ("dx",))
    zero = _run(dict(a, d_out=torch.zeros_like(a["d_out"])), "none", ws)
    assert not any(bool(t.any()) for t in zero.values())
    none = _run(dict(a, x=a["x"][:0], d_out=a["d_out"][:0]), "none", ws.fill_(255))
    assert not none["dw"].any() and not none["dbias"].any()
    # an infinity and a NaN stay in their row of dx, and the others keep their accuracy
    bad = a["d_out"].clone()
    bad[3, 7], bad[99, 0] = float("inf"), float("nan")
    got = _run(dict(a, d_out=bad), "none", ws)
    rows = [r for r in range(130) if r not in (3, 99)]
    assert not torch.isfinite(got["dx"][[3, 99]]).any()
    assert torch.equal(got["dx"][rows], whole["dx"][rows])
    assert not torch.isfinite(got["dw"][[0, 7]]).any() and torch.isfinite(got["dw"][1:7]).all()


def test_parts_and_replays():
    """dx and dw alone are those of the whole call; a captured call follows
    gradients that grow and shrink between its replays."""
    m = _m()
    a = _inputs(640, 60, 1032, "swiglu", F32, 8, 2.0 ** -22, 256.0, 2048.0)
    whole = _run(a, "swiglu")
    for name in ("dx", "dw"):
        one = {name: torch.empty_like(whole[name])}
        m.moe_linear_backward(a["x"], a["w"], a["d_out"], pre=a["pre"], act=m.ACT_SWIGLU, **one)
        assert torch.equal(one[name], whole[name])
    dx, dw = torch.empty_like(a["x"]), torch.empty_like(a["w"])
    call = lambda: m.moe_linear_backward(a["x"], a["w"], a["d_out"], pre=a["pre"], act=m.ACT_SWIGLU, dx=dx, dw=dw)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for e in (0, 6, -5, 3, -12):
        a["d_out"].mul_(2.0 ** e)
        call()
        torch.cuda.synchronize()
        want = dx.clone(), dw.clone()
        dx.fill_(5.0), dw.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]), e
        _check(a, "swiglu", dict(_run(a, "swiglu"), dx=dx, dw=dw))


@pytest.mark.parametrize("what,M,N,K", [c for c in EACH_TILE if c[0] in ("dx", "dw")])
def test_every_tile_of_the_gradients(what, M, N, K):
    """Each tile, whole and split: the factor is taken off in the tiles'
    epilogue and in the join.  The reference is float64 on the GPU."""
    m = _m()
    say(f"[linear range] {what} {M}x{N}x{K}")
    size = 2.0 ** -26
    terms = M if what == "dw" else N
    s = min(2.0 ** 12, 2.0 ** 4 / (size * terms))
    a = _inputs(M, N, K, "none", F32, M + K, size, s, s)
    g, x, w = a["d_out"].double(), a["x"].double(), a["w"].double()
    # (all terms are positive: the sum of magnitudes is the sum)
    if what == "dx":
        got, ref = torch.empty_like(a["x"]), torch.mm(g, w)
        m.moe_linear_backward(a["x"], a["w"], a["d_out"], dx=got)
        tail = 2.0 ** -39 * g.max() * w.sum(0, keepdim=True)
    else:
        got, ref = torch.empty_like(a["w"]), torch.mm(g.t().contiguous(), x)
        m.moe_linear_backward(a["x"], a["w"], a["d_out"], dw=got)
        tail = 2.0 ** -39 * g.max() * x.sum(0, keepdim=True)
    err = HALF * ref + tail + (terms + 64) * U * (1 + HALF) * ref
    bound = err * (1 + HALF) + HALF * ref + 2.0 ** -25
    assert bool(((got.double() - ref).abs() <= bound).all())
    assert float(ref.max()) > 2.0 ** -14 and float(ref.max()) < 65504
