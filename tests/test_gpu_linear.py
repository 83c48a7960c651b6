"""The dense product and its gradients on the GPU against the float64 oracle.

Tolerances are bounds, not fits.  With u = 2^-24 and S = |x| |w|^T + |b|, an
fp32 sum of depth exact products is off by at most (depth + 2) u S whatever its
order.  An activation passes an error on with its largest slope (1.13 for the
smooth ones here) and adds a few u of its value (8 u, and 64 u |z| where exp
takes a rounded argument); a gated one multiplies the two halves' errors by the
other half.  Every 16-bit result adds half a step, eps / 2 of its value.  In
the gradients each dz is rounded to 16 bits, eps / 2 |dz|, which a product sums
as eps / 2 |dz| |w|.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import linear as OL

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _m():
    import moe_expert_tile_amd as m
    return m


def _act(name):
    return getattr(_m(), "ACT_" + name.upper())


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _tiny(dtype):
    return 2.0 ** -25 if dtype is torch.float16 else 2.0 ** -140


def _inputs(M, N, K, act, dtype, seed, bias=True, residual=True, out="same"):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=DT[dtype]):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    n = 2 * N if act == "swiglu" else N
    o = DT[dtype] if out == "same" else torch.float32
    return dict(x=randn(M, K), w=randn(n, K, std=K ** -0.5), bias=randn(n, std=0.5) if bias else None,
                residual=randn(M, N, dtype=o) if residual else None, d_out=randn(M, N, dtype=o),
                out=torch.full((M, N), float("nan"), dtype=o, device="cuda"),
                pre=torch.full((M, n), float("nan"), dtype=DT[dtype], device="cuda"))


def _forward_error(x, w, b, act, z):
    """(bound on z's error, bound on the activation's error)"""
    S = np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(b))
    ez = (x.shape[1] + 2) * U * S
    if act == "swiglu":
        n = z.shape[1] // 2
        g, u = z[:, :n], z[:, n:]
        sg = np.abs(OL.activation("silu", g))
        own = (16 * U + 64 * U * np.abs(g)) * sg * np.abs(u)
        return ez, 1.13 * ez[:, :n] * np.abs(u) + sg * ez[:, n:] + 1.13 * ez[:, :n] * ez[:, n:] + own
    y = np.abs(OL.activation(act, z))
    if act in ("none", "relu"):
        return ez, ez
    return ez, 1.13 * ez + 16 * U * np.abs(z) + 64 * U * np.abs(z) * y


def _check_forward(a, act, ws=None):
    m = _m()
    res = None if a["residual"] is None else a["residual"].clone()
    m.moe_linear(a["x"], a["w"], a["out"], bias=a["bias"], residual=a["residual"], pre=a["pre"], act=_act(act), ws=ws)
    torch.cuda.synchronize()
    x, w, b = _np(a["x"]), _np(a["w"]), _np(a["bias"])
    z = OL.product(x, w, b)
    ez, ey = _forward_error(x, w, b, act, z)
    r = 0 if res is None else _np(res)
    y = OL.apply(act, z) + r
    half = _half(a["out"].dtype)
    err = np.abs(_np(a["out"]) - y)
    bound = (ey + U * (np.abs(y) + np.abs(r))) * (1 + half) + half * np.abs(y) + _tiny(a["out"].dtype)
    assert np.all(err <= bound), (err - bound).max()
    if a["pre"] is not None:
        half = _half(a["pre"].dtype)
        err = np.abs(_np(a["pre"]) - z)
        assert np.all(err <= ez * (1 + half) + half * np.abs(z) + _tiny(a["pre"].dtype))


# every tile, edges of each, sums from one chunk to several splits
SIZES = [(1, 1, 8), (1, 7168, 2048), (1, 250, 7168), (3, 40, 8200), (20, 256, 7176), (32, 1030, 4096), (2, 16, 64), (7, 33, 40), (16, 100, 512), (17, 60, 256), (31, 48, 1000),
         (33, 130, 72), (64, 64, 64), (65, 60, 512), (65, 1, 8), (100, 256, 4096), (128, 128, 128), (129, 513, 264),
         (200, 60, 2056), (257, 255, 192), (300, 1000, 8), (512, 256, 1024), (1000, 130, 136), (2049, 516, 328),
         (4100, 2052, 72)]


@pytest.mark.parametrize("act", ["none", "swiglu", "gelu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(M, N, K, act):
    if M * N > 1 << 22 and act != "none":
        N //= 4
    for dtype, out in (("bf16", "same"), ("f16", "f32")):
        say(f"[linear] {M}x{N}x{K} {act} {dtype} {out}")
        _check_forward(_inputs(M, N, K, act, dtype, M + N, out=out), act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "same")])
def test_activations_and_options(act, dtype, out):
    for M, N, K in ((5, 44, 96), (150, 90, 136)):
        for bias in (False, True):
            for residual in (False, True):
                a = _inputs(M, N, K, act, dtype, 3, bias=bias, residual=residual, out=out)
                a["w"] *= 3        # sums out where the activations bend
                _check_forward(a, act)
                a["pre"] = None
                _check_forward(a, act)


@pytest.mark.parametrize("M,N,K", [(300, 520, 200), (1100, 264, 2056), (520, 512, 520)])
def test_large_tiles_of_every_kind(M, N, K):
    """Sizes below one 256-row tile's worth of work choose small tiles; these
    are repeated on a batch large enough for the others."""
    for act in ("none", "swiglu", "silu"):
        for scale in (1, 6):
            a = _inputs(M * scale, N, K, act, "bf16", 5)
            _check_forward(a, act)


def _strided(t, pad, fill=float("nan")):
    if t is None:
        return None
    big = torch.full((t.shape[0] * 2, t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    view = big[::2, :t.shape[1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("M,N,K", [(9, 37, 72), (140, 61, 136), (600, 300, 520)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_strides(M, N, K, act):
    """Row pitches beyond the rows' length: what lies between is not read into
    the sums and not written."""
    a = _inputs(M, N, K, act, "bf16", 9)
    packed = dict(a, out=a["out"].clone(), pre=a["pre"].clone())
    _check_forward(packed, act)
    s = {k: _strided(v, 8 if k in ("x", "w") else 3) if v is not None and v.dim() == 2 else v for k, v in a.items()}
    s["bias"] = a["bias"]
    keep_out, keep_pre = s["out"]._base.clone(), s["pre"]._base.clone()
    _check_forward(s, act)
    assert torch.equal(s["out"], packed["out"]) and torch.equal(s["pre"], packed["pre"])
    for view, was in ((s["out"], keep_out), (s["pre"], keep_pre)):
        now = view._base.clone()
        now[::2, :view.shape[1]] = was[::2, :view.shape[1]]
        assert torch.equal(now.isnan(), was.isnan())


def test_residual_in_place_and_workspace():
    m = _m()
    for M, N, K in ((3, 256, 512), (128, 64, 8192), (512, 512, 256)):
        a = _inputs(M, N, K, "none", "bf16", 21)
        a["pre"] = None
        m.moe_linear(a["x"], a["w"], a["out"], bias=a["bias"], residual=a["residual"])
        d = m.moe_linear_desc(M, N, K, 0, 0, 0, 0)
        need = m.moe_linear_sizes(d)["forward_bytes"]
        ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")   # NaNs: its contents do not matter
        run = a["residual"].clone()
        m.moe_linear(a["x"], a["w"], run, bias=a["bias"], residual=run, ws=ws)
        assert torch.equal(run, a["out"])
        assert bool((ws[need:] == 255).all())
        if need:
            with pytest.raises(m.MoEError):
                m.moe_linear(a["x"], a["w"], run, ws=ws[:need - 1])


def test_infinities_stay_in_their_rows():
    m = _m()
    for M in (5, 200):
        a = _inputs(M, 96, 136, "none", "bf16", 2)
        a["x"][3, 7] = float("inf")
        a["x"][4, 8] = float("nan")
        m.moe_linear(a["x"], a["w"], a["out"])
        bad = (~torch.isfinite(a["out"])).any(1)
        assert bad.nonzero().flatten().tolist() == [3, 4]


def test_no_rows():
    m = _m()
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.randn(32, 64, device="cuda").to(torch.bfloat16)
    m.moe_linear(x, w, torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"))
    dw, db = torch.full_like(w, 5.0), torch.full((32,), 5.0, dtype=torch.bfloat16, device="cuda")
    m.moe_linear_backward(x, w, torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), dx=torch.empty_like(x), dw=dw,
                          dbias=db)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_one_gradient_alone_without_rows(act):
    """An empty dx is given, though its address is 0 (a frozen expert without rows)."""
    m = _m()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    n = 64 if act == "swiglu" else 32
    x, w, g, pre = torch.empty(0, 64, **bf), torch.ones(n, 64, **bf), torch.empty(0, 32, **bf), torch.empty(0, n, **bf)
    m.moe_linear_backward(x, w, g, dx=torch.empty_like(x), pre=pre, act=_act(act))
    db = torch.full((n,), 5.0, **bf)
    m.moe_linear_backward(x, w, g, dbias=db, pre=pre, act=_act(act))
    assert not db.any()


# --- gradients -------------------------------------------------------------------

def _check_backward(a, act, want=("dx", "dw", "dbias"), place=None):
    m = _m()
    x, w, g = _np(a["x"]), _np(a["w"]), _np(a["d_out"])
    n = a["w"].shape[0]
    dtype = a["x"].dtype
    got = {"dx": torch.full_like(a["x"], 9.0), "dw": torch.full_like(a["w"], 9.0),
           "dbias": torch.full((n,), 9.0, dtype=dtype, device="cuda")}
    got = {k: v for k, v in got.items() if k in want}
    if place:
        got.update(place)
    m.moe_linear_backward(a["x"], a["w"], a["d_out"], pre=a["pre"], act=_act(act), **got)
    torch.cuda.synchronize()
    pre = None if act == "none" else _np(a["pre"])
    dz = OL.dz(act, g, pre)
    half = _half(dtype)
    # dz's own error: slopes (and silu's values) to a few u, exp's argument rounded
    if act == "none":
        e32 = 0 * np.abs(dz)
    elif act == "swiglu":
        z = np.abs(pre)
        gu = np.concatenate([np.abs(g * pre[:, g.shape[1]:]), np.abs(g * pre[:, :g.shape[1]])], 1)
        e32 = (16 + 64 * np.concatenate([z[:, :g.shape[1]]] * 2, 1)) * U * gu
    else:
        e32 = (16 + 64 * np.abs(pre) * (1 + pre ** 2)) * U * np.abs(g)
    edz = half * np.abs(dz) + (1 + half) * e32 + _tiny(dtype)
    for name, ref, err in (("dx", dz @ w, edz @ np.abs(w) + (n + 8) * U * (np.abs(dz) + edz) @ np.abs(w)),
                           ("dw", dz.T @ x, edz.T @ np.abs(x) + (len(x) + 64) * U * (np.abs(dz) + edz).T @ np.abs(x)),
                           ("dbias", dz.sum(0), (e32 + (len(x) + 2) * U * np.abs(dz)).sum(0))):
        if name in got:
            d = np.abs(_np(got[name]) - ref)
            bound = err * (1 + half) + half * np.abs(ref) + _tiny(dtype)
            assert np.all(d <= bound), (name, (d - bound).max())
    return got


@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (1, 64, 128), (3, 31, 40), (64, 60, 512), (65, 63, 72), (100, 65, 200),
                                   (130, 128, 264), (257, 100, 1000), (512, 60, 2048), (1025, 520, 328),
                                   (4097, 257, 136)])
@pytest.mark.parametrize("act", ["none", "swiglu", "silu"])
def test_backward(M, N, K, act):
    for dtype, out in (("bf16", "same"), ("f16", "f32")):
        say(f"[linear back] {M}x{N}x{K} {act} {dtype} {out}")
        a = _inputs(M, N, K, act, dtype, M + N, out=out)
        a["pre"].normal_(generator=torch.Generator(device="cuda").manual_seed(4))
        if act == "none":
            a["pre"] = None
        _check_backward(a, act)


@pytest.mark.parametrize("act", ACTS)
def test_backward_of_every_activation_and_part(act):
    a = _inputs(150, 72, 136, act, "bf16", 6)
    a["pre"].normal_(std=2.0)
    a["pre"][0, :6] = torch.tensor([0.0, -0.0, 30.0, -30.0, 120.0, -120.0])
    whole = _check_backward(a, act)
    for want in (("dx",), ("dw",), ("dbias",), ("dx", "dw")):
        part = _check_backward(a, act, want)
        for k in want:
            assert torch.equal(part[k], whole[k]), (want, k)


def test_backward_strides():
    a = _inputs(140, 61, 136, "swiglu", "bf16", 8)
    a["pre"].normal_()
    whole = _check_backward(a, "swiglu")
    s = {k: _strided(v, 8 if k in ("x", "w") else 3) if v is not None and v.dim() == 2 else v for k, v in a.items()}
    place = {"dx": _strided(whole["dx"] * 0, 5), "dw": _strided(whole["dw"] * 0, 7)}
    got = _check_backward(s, "swiglu", place=place)
    for k in whole:
        assert torch.equal(got[k], whole[k])
    for k in ("dx", "dw"):
        rest = got[k]._base.clone()
        rest[::2, :got[k].shape[1]] = float("nan")
        assert bool(rest.isnan().all())


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_backward_without_x_or_w(act):
    """What a gradient does not need may be missing (through the C entry point)."""
    import ctypes
    m = _m()
    a = _inputs(70, 40, 64, act, "bf16", 10)
    a["pre"].normal_()
    whole = _check_backward(dict(a, pre=a["pre"] if act != "none" else None), act)
    d = m.moe_linear_desc(70, 40, 64, 0, 0, _act(act), 0)
    ws = torch.empty(m.moe_linear_sizes(d)["backward_bytes"], dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    dx, dw = torch.zeros_like(a["x"]), torch.zeros_like(a["w"])
    p = lambda t: t.data_ptr()  # noqa: E731
    assert m._lib.moe_linear_backward(ctypes.byref(d), None, p(a["w"]), p(a["pre"]), p(a["d_out"]), p(dx), None, None, p(ws), s) == 0
    assert m._lib.moe_linear_backward(ctypes.byref(d), p(a["x"]), None, p(a["pre"]), p(a["d_out"]), None, p(dw), None, p(ws), s) == 0
    torch.cuda.synchronize()
    assert torch.equal(dx, whole["dx"]) and torch.equal(dw, whole["dw"])


def test_offsets_beyond_32_bits():
    """2^21 rows of 1032 columns are 2.16e9 elements: the first and the last
    rows' results are those of small calls on copies of them."""
    m = _m()
    M, K, N = 1 << 21, 1032, 8
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").fill_(0.25)
    w = torch.randn(N, K, device="cuda").to(torch.bfloat16)
    ends = (slice(0, 200), slice(M - 200, M))
    for e in ends:
        x[e] = torch.randn(200, K, device="cuda").to(torch.bfloat16)
    out, g = torch.empty(M, N, device="cuda"), torch.zeros(M, N, device="cuda")
    for e in ends:
        g[e] = torch.randn(200, N, device="cuda")
    say("[linear] 2^21 rows")
    m.moe_linear(x, w, out)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    say("[linear back] 2^21 rows")
    m.moe_linear_backward(x, w, g, dx=dx, dw=dw)
    torch.cuda.synchronize()
    S = 0
    for e in ends:
        xe = _np(x[e])
        z = xe @ _np(w).T
        assert np.all(np.abs(_np(out[e]) - z) <= (K + 2) * U * (np.abs(xe) @ np.abs(_np(w)).T))
        small = torch.empty(200, K, dtype=torch.bfloat16, device="cuda")
        m.moe_linear_backward(x[e].contiguous(), w, g[e].contiguous(), dx=small)
        assert torch.equal(small, dx[e])
        S = S + _np(g[e]).T @ xe
    assert not dx[1000:1100].any()
    mag = sum(np.abs(_np(g[e])).T @ np.abs(_np(x[e])) for e in ends)
    half = _half(torch.bfloat16)
    assert np.all(np.abs(_np(dw) - S) <= half * 1.01 * (mag + np.abs(S)) + 2.0 ** -20)


# Ragged sizes whose work asks for each tile (64, 128 and 256 rows), whole and
# split along the sum, in each direction; the reference is float64 on the GPU.
EACH_TILE = [
    ("fwd", 101, 11, 1752), ("fwd", 648, 8838, 144), ("fwd", 3417, 9, 5112), ("fwd", 1665, 7185, 144),
    ("fwd", 8880, 132, 7376), ("gated", 86, 6, 496), ("gated", 101, 6, 1752), ("gated", 648, 4420, 144),
    ("gated", 3417, 5, 5112), ("gated", 1665, 3593, 144), ("gated", 8880, 67, 7376),
    ("dx", 535, 182, 8), ("dx", 104, 1502, 8), ("dx", 4551, 149, 1304), ("dx", 3111, 5106, 8), ("dx", 1707, 142, 7216),
    ("dx", 8623, 7572, 136), ("dw", 467, 44, 16), ("dw", 1618, 12, 8), ("dw", 143, 6333, 912), ("dw", 2350, 6271, 8),
    ("dw", 141, 2961, 4280), ("dw", 7852, 8460, 136),
    # the 128 x 256 tile with its three stages: whole, and splits that end with 1, 2 and more stages
    ("fwd", 459, 8251, 328), ("fwd", 2065, 134, 8472), ("fwd", 2636, 145, 8560), ("fwd", 2834, 130, 3904),
    ("gated", 3022, 650, 336), ("gated", 2087, 70, 8480), ("gated", 71, 2412, 8576), ("gated", 70, 5517, 1808),
    ("dx", 8861, 327, 416), ("dx", 2073, 8460, 184), ("dx", 2793, 3937, 136),
    ("dw", 337, 9480, 416), ("dw", 7812, 2131, 136), ("dw", 2988, 69, 8416),
    # the others split (and 64 rows whole)
    ("fwd", 40, 2, 8), ("fwd", 4500, 2, 3592), ("fwd", 8253, 394, 3712), ("gated", 6777, 2, 2032),
    ("gated", 206, 8224, 3448), ("dx", 8343, 1848, 8), ("dx", 6726, 3380, 536), ("dx", 2085, 5704, 136),
    ("dw", 4252, 8292, 392), ("dw", 3606, 66, 5648),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("what,M,N,K", EACH_TILE)
def test_every_tile_whole_and_split(what, M, N, K, dtype):
    m = _m()
    say(f"[linear tiles] {what} {M}x{N}x{K} {dtype}")
    a = _inputs(M, N, K, "swiglu" if what == "gated" else "none", dtype, M + K)
    x, w, half, tiny = a["x"].double(), a["w"].double(), _half(DT[dtype]), _tiny(DT[dtype])
    if what in ("fwd", "gated"):
        b, r = a["bias"].double(), a["residual"].double()
        m.moe_linear(a["x"], a["w"], a["out"], bias=a["bias"], residual=a["residual"], pre=a["pre"],
                     act=_act("swiglu" if what == "gated" else "none"))
        z = torch.mm(x, w.t().contiguous()) + b
        ez = (K + 2) * U * (torch.mm(x.abs(), w.abs().t().contiguous()) + b.abs())
        if what == "gated":
            g, u = z[:, :N], z[:, N:]
            p = torch.sigmoid(g)
            sg = (g * p).abs()
            y = g * p * u
            ey = (1.13 * ez[:, :N] * u.abs() + sg * ez[:, N:] + 1.13 * ez[:, :N] * ez[:, N:] +
                  (16 * U + 64 * U * g.abs()) * sg * u.abs())
        else:
            y, ey = z, ez
        y = y + r
        bound = (ey + U * (y.abs() + r.abs())) * (1 + half) + half * y.abs() + tiny
        assert bool(((a["out"].double() - y).abs() <= bound).all())
        assert bool(((a["pre"].double() - z).abs() <= ez * (1 + half) + half * z.abs() + tiny).all())
        return
    g = a["d_out"].double()
    if what == "dx":
        got = torch.empty_like(a["x"])
        m.moe_linear_backward(a["x"], a["w"], a["d_out"], dx=got)
        ref, mag, terms = torch.mm(g, w), torch.mm(g.abs(), w.abs()), N
    else:
        got = torch.empty_like(a["w"])
        m.moe_linear_backward(a["x"], a["w"], a["d_out"], dw=got)
        ref, mag, terms = torch.mm(g.t().contiguous(), x), torch.mm(g.t().contiguous().abs(), x.abs()), M
    bound = (terms + 64) * U * mag * (1 + half) + half * ref.abs() + tiny
    assert bool(((got.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("M", [2, 40])
def test_a_vocabulary_of_columns(M):
    """Far more columns than rows: 200003 of them, an odd number."""
    a = _inputs(M, 200003, 64, "none", "bf16", 12)
    _m().moe_linear(a["x"], a["w"], a["out"], bias=a["bias"], residual=a["residual"])
    z = torch.mm(a["x"].double(), a["w"].double().t().contiguous()) + a["bias"].double()
    y = z + a["residual"].double()
    S = torch.mm(a["x"].double().abs(), a["w"].double().abs().t().contiguous()) + a["bias"].double().abs()
    bound = (66 * U * S + U * (y.abs() + a["residual"].double().abs())) * 1.01 + _half(torch.bfloat16) * y.abs()
    assert bool(((a["out"].double() - y).abs() <= bound).all())
    got = _check_backward(dict(a, pre=None, w=a["w"][:4099], d_out=a["d_out"][:, :4099].contiguous()), "none")
    assert got["dw"].shape == (4099, 64)
