"""The dense product's epilogue on every tile of the many-row kernel: without
an activation and a kept pre-activation (a branch of its own: all residual
reads ahead of the stores), and with the residual added in place.

References are float64 on the GPU, bounds those of test_gpu_linear.py."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_linear import DT, U, _act, _half, _inputs, _m, _tiny

pytestmark = pytest.mark.gpu

# (columns odd or not of whole 8s, and of whole 8s) for the tiles of 64 x 128, 128 x 128, 256 x 256 and 128 x 256,
# whole and split
SIZES = [(40, 2, 8), (40, 8, 8), (101, 11, 1752), (101, 16, 1752), (648, 8838, 144), (648, 8840, 144), (3417, 9, 5112),
         (3417, 8, 5112), (1665, 7185, 144), (1665, 7184, 144), (8253, 394, 3712), (8253, 392, 3712), (459, 8251, 328),
         (459, 8256, 328), (2065, 134, 8472), (2065, 136, 8472)]
# ... and gated
GATED = [(86, 6, 496), (101, 8, 1752), (648, 4420, 144), (3417, 5, 5112), (1665, 3593, 144), (1665, 3592, 144),
         (206, 8224, 3448), (3022, 650, 336), (70, 5517, 1808)]


def _z(a):
    x, w = a["x"].double(), a["w"].double()
    z = torch.mm(x, w.t().contiguous())
    mag = torch.mm(x.abs(), w.abs().t().contiguous())
    if a["bias"] is not None:
        z += a["bias"].double()
        mag += a["bias"].double().abs()
    return z, (a["x"].shape[1] + 2) * U * mag


def _close(out, y, ey, res):
    half = _half(out.dtype)
    r = 0 if res is None else res.double()
    y = y + r
    bound = (ey + U * (y.abs() + (r.abs() if res is not None else 0))) * (1 + half) + half * y.abs() + _tiny(out.dtype)
    return bool(((out.double() - y).abs() <= bound).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_without_activation_and_pre(M, N, K, dtype):
    m = _m()
    for out in ("same", "f32"):
        a = _inputs(M, N, K, "none", dtype, M + N, out=out)
        z, ez = _z(a)
        bare, ebare = _z(dict(a, bias=None))
        for bias, res in ((True, True), (False, True), (True, False), (False, False)):
            say(f"[linear epilogue] {M}x{N}x{K} {dtype} {out} bias={bias} residual={res}")
            a["out"].fill_(float("nan"))
            m.moe_linear(a["x"], a["w"], a["out"], bias=a["bias"] if bias else None,
                         residual=a["residual"] if res else None)
            r = a["residual"] if res else None
            assert _close(a["out"], z if bias else bare, ez if bias else ebare, r)
        # in place: the same bits
        m.moe_linear(a["x"], a["w"], a["out"], bias=a["bias"], residual=a["residual"])
        run = a["residual"].clone()
        m.moe_linear(a["x"], a["w"], run, bias=a["bias"], residual=run)
        assert torch.equal(run, a["out"])


@pytest.mark.parametrize("act,M,N,K", [("silu", *s) for s in SIZES] + [("swiglu", *s) for s in GATED])
def test_in_place_under_an_activation(act, M, N, K):
    m = _m()
    for dtype, out, keep in (("bf16", "same", False), ("f16", "f32", True)):
        say(f"[linear epilogue] {M}x{N}x{K} {act} {dtype} {out} in place")
        a = _inputs(M, N, K, act, dtype, M + N, out=out)
        if not keep:
            a["pre"] = None
        z, ez = _z(a)
        run = a["residual"].clone()
        m.moe_linear(a["x"], a["w"], run, bias=a["bias"], residual=run, pre=a["pre"], act=_act(act))
        if act == "swiglu":
            g, u = z[:, :N], z[:, N:]
            y = g * torch.sigmoid(g) * u
            sg = (g * torch.sigmoid(g)).abs()
            ey = (1.13 * ez[:, :N] * u.abs() + sg * ez[:, N:] + 1.13 * ez[:, :N] * ez[:, N:] +
                  (16 * U + 64 * U * g.abs()) * sg * u.abs())
        else:
            y = z * torch.sigmoid(z)
            ey = 1.13 * ez + 16 * U * z.abs() + 64 * U * z.abs() * y.abs()
        assert _close(run, y, ey, a["residual"])
        if keep:
            half = _half(DT[dtype])
            assert bool(((a["pre"].double() - z).abs() <= ez * (1 + half) + half * z.abs() + _tiny(DT[dtype])).all())


@pytest.mark.parametrize("M,N,K", [(1665, 7184, 144), (459, 8251, 328)])
def test_strided_residual_in_place(M, N, K):
    """The residual and output as one view of wider rows: the rest stays."""
    m = _m()
    a = _inputs(M, N, K, "none", "bf16", 3)
    m.moe_linear(a["x"], a["w"], a["out"], bias=a["bias"], residual=a["residual"])
    wide = torch.full((M, N + 13), 7.0, dtype=torch.bfloat16, device="cuda")
    view = wide[:, 5:5 + N]
    view.copy_(a["residual"])
    m.moe_linear(a["x"], a["w"], view, bias=a["bias"], residual=view)
    assert torch.equal(view, a["out"])
    assert bool((wide[:, :5] == 7).all()) and bool((wide[:, 5 + N:] == 7).all())
