"""Microscaled 4-bit rows on the GPU: quantisation and its inverse bit by bit,
and the product with 4-bit weights against the float64 oracle, from one row of
one expert to long ragged batches.

The products' tolerances are those of the dense product: with u = 2^-24 and S =
|x| |w|^T + |b|, an fp32 sum of exact products is off by at most (depth + 2) u S.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import linear as OL
from oracle import mx as OM
from test_gpu_linear import _forward_error

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _m():
    import moe_expert_tile_amd as m
    return m


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _bytes(t):
    return t.cpu().numpy()


def _quantize(x, **kw):
    m = _m()
    M, K = x.shape
    q = torch.full((M, K // 2), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((M, K // 32), 77, dtype=torch.uint8, device="cuda")
    m.moe_mx_quantize(x, q, s, **kw)
    return q, s


# --- quantisation ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,K", [(1, 32), (1, 64), (3, 96), (7, 2048), (33, 160), (2, 7168), (129, 256)])
def test_quantize_and_back(M, K, dtype):
    m = _m()
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn(M, K, generator=gen, device="cuda") * torch.exp(3 * torch.randn(M, K // 32, generator=gen, device="cuda")).repeat_interleave(32, 1)
    x[:, ::7] = 0
    x = x.to(DT[dtype])
    q, s = _quantize(x)
    want = OM.quantize(_np(x))
    assert np.array_equal(_bytes(q), want[0]) and np.array_equal(_bytes(s), want[1])
    for out in DT.values():
        back = torch.full((M, K), 9.0, dtype=out, device="cuda")
        m.moe_mx_dequantize(q, s, back)
        assert torch.equal(back, torch.from_numpy(OM.values(*want)).cuda().to(out))


@pytest.mark.parametrize("dtype", list(DT))
def test_every_value_of_a_type(dtype):
    """Each 16-bit pattern beside a power of two that sets the block's scale (fp32: the patterns next to ties)."""
    if dtype == "f32":
        ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7.99], np.float32).view(np.int32)
        bits = np.concatenate([(ties + d).astype(np.int32) for d in (-2, -1, 0, 1, 2)])
        v = torch.from_numpy(np.concatenate([bits.view(np.float32), -bits.view(np.float32)]))
        v = torch.cat([v * 2.0 ** e for e in (-149, -127, -126, -60, 0, 60, 124)])
        tops = [4.0 * 2.0 ** e for e in (-149, -127, -126, -60, 0, 60, 124)]
    else:
        v = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16)).view(DT[dtype])
        v = v[torch.isfinite(v)]
        tops = [2.0 ** -20, 4.0, 2.0 ** 12] + ([2.0 ** -126, 2.0 ** 100] if dtype == "bf16" else [2.0 ** -24])
    v = v[:v.numel() // 31 * 31].view(-1, 31)
    x = torch.cat([torch.cat([torch.full((v.shape[0], 1), t, dtype=DT[dtype]), v.to(DT[dtype])], 1) for t in tops])
    q, s = _quantize(x.cuda())
    want = OM.quantize(_np(x))
    assert np.array_equal(_bytes(s), want[1]) and np.array_equal(_bytes(q), want[0])


@pytest.mark.parametrize("dtype", list(DT))
def test_blocks_that_are_not_numbers_and_empty_ones(dtype):
    x = torch.randn(4, 128, device="cuda").to(DT[dtype])
    x[0, 5] = float("inf")
    x[1, 40] = float("nan")
    x[2, 64:96] = 0
    x[3, 127] = float("-inf")
    q, s = _quantize(x)
    want = OM.quantize(_np(x))
    assert np.array_equal(_bytes(q), want[0]) and np.array_equal(_bytes(s), want[1])
    assert int((s == 255).sum()) == 3 and int(s[2, 2]) == 0
    out = torch.empty(4, 128, device="cuda")
    _m().moe_mx_dequantize(q, s, out)
    bad = torch.isnan(out).view(4, 4, 32)
    assert torch.equal(bad.all(2), s == 255) and torch.equal(bad.any(2), s == 255)


def test_dequantize_every_byte_and_scale():
    m = _m()
    q = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 256).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1).repeat(1, 16)
    want = torch.from_numpy(OM.values(_bytes(q), _bytes(s)))
    for dtype in DT.values():
        out = torch.empty(256, 512, dtype=dtype, device="cuda")
        m.moe_mx_dequantize(q, s, out)
        # float64 to bf16 rounds through fp32 here, which holds every value that is in range
        ref = want.to(torch.float32).to(dtype)
        got = out.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got.nan_to_num(nan=0.0, posinf=float("inf"), neginf=-float("inf")),
                           ref.nan_to_num(nan=0.0, posinf=float("inf"), neginf=-float("inf")))


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_pitches(dtype):
    """Rows apart from each other and off 16 bytes: what lies between is neither read nor written."""
    m = _m()
    M, K = 37, 224
    big = torch.full((M, K + 13), float("nan"), dtype=DT[dtype], device="cuda")
    x = big[:, 3:3 + K]
    x.copy_(torch.randn(M, K, device="cuda"))
    qb, sb = torch.full((M, K // 2 + 16), 77, dtype=torch.uint8, device="cuda"), torch.full((M, K // 32 + 3), 77, dtype=torch.uint8, device="cuda")
    m.moe_mx_quantize(x, qb[:, :K // 2], sb[:, 1:1 + K // 32])
    want = OM.quantize(_np(x))
    assert np.array_equal(_bytes(qb[:, :K // 2]), want[0]) and np.array_equal(_bytes(sb[:, 1:1 + K // 32]), want[1])
    assert bool((qb[:, K // 2:] == 77).all()) and bool((sb[:, 0] == 77).all()) and bool((sb[:, 1 + K // 32:] == 77).all())
    out = torch.full_like(big, 9.0)
    m.moe_mx_dequantize(qb[:, :K // 2], sb[:, 1:1 + K // 32], out[:, 3:3 + K])
    assert torch.equal(out[:, 3:3 + K], torch.from_numpy(OM.values(*want)).cuda().to(DT[dtype]))
    assert bool((out[:, :3] == 9).all()) and bool((out[:, 3 + K:] == 9).all())


def test_quantize_many_and_none():
    m = _m()
    none = torch.empty(0, 64, device="cuda")
    m.moe_mx_quantize(none, torch.empty(0, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(70000, 32, generator=gen, device="cuda")          # more rows than a grid has
    big = torch.zeros(70000, 48, device="cuda")
    big[:, :32] = x
    q, s = _quantize(x)
    q2, s2 = _quantize(big[:, :32])
    assert torch.equal(q, q2) and torch.equal(s, s2)
    pick = [0, 4095, 4096, 69999]
    want = OM.quantize(_np(x[pick]))
    assert np.array_equal(_bytes(q[pick]), want[0]) and np.array_equal(_bytes(s[pick]), want[1])
    # over 2^32 bytes
    y = torch.zeros(1 << 20, 4128, dtype=torch.bfloat16, device="cuda")
    y[-1] = torch.randn(4128, generator=gen, device="cuda")
    q, s = _quantize(y)
    want = OM.quantize(_np(y[-1:]))
    assert np.array_equal(_bytes(q[-1:]), want[0]) and np.array_equal(_bytes(s[-1:]), want[1])
    assert not bool(q[:-1].any())


# --- product ------------------------------------------------------------------------

def _offsets(M, E, kind, rng):
    """Each expert's first row: rows shared out evenly, with one loud expert, to a few experts alone, or apart from
    the buffer's ends."""
    if kind == "even":
        return np.linspace(0, M, E + 1).astype(np.int32)
    if kind == "ends":
        inner = np.sort(rng.integers(M // 5, M - M // 7 + 1, E + 1))
        return inner.astype(np.int32)
    p = np.where(rng.random(E) < 0.5, 0.0, rng.random(E)) if kind == "few" else 1.0 / (1 + np.arange(E)) ** 1.5
    if p.sum() == 0:
        p[E // 2] = 1
    return np.concatenate([[0], np.cumsum(rng.multinomial(M, p / p.sum()))]).astype(np.int32)


def _weights(E, n, K, gen, spread=0):
    """Codes and scales as a quantiser gives them, scales over a wider range with `spread`."""
    q = torch.randint(0, 256, (E, n, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.randint(118 - spread, 122 + spread, (E, n, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return q, s


def _check(M, N, K, E, act, xt, out_t, kind="even", bias=False, spread=0, seed=0, pitches=False, offsets=True, stream=None):
    m = _m()
    say(f"[mx linear] {M}x{N}x{K} E={E} {kind} {act} {xt} -> {out_t} bias={bias} pitches={pitches}")
    gen = torch.Generator(device="cuda").manual_seed(seed + M + N + K)
    rng = np.random.default_rng(seed + M + N + K)
    n = 2 * N if act == "swiglu" else N
    off = _offsets(M, E, kind, rng) if offsets else np.array([0, M], np.int32)
    q, s = _weights(E, n, K, gen, spread)
    w = OM.values(_bytes(q), _bytes(s))
    x = torch.randn(M, K, generator=gen, device="cuda")
    held = np.zeros(M, bool)
    for e in range(E):
        held[off[e]:off[e + 1]] = True
    if xt == "mx":
        xq, xs = _quantize(x)
        xs[torch.from_numpy(~held).cuda()] = 255                   # rows of no expert do not matter
        xr = np.nan_to_num(OM.values(_bytes(xq), _bytes(xs)))
        if pitches:
            xq, xs = _apart(xq, 32), _apart(xs, 5, 3)
        args = dict(x=xq, x_scale=xs)
    else:
        x = x.to(DT[xt])
        x[torch.from_numpy(~held).cuda()] = float("nan")
        xr = np.nan_to_num(_np(x))
        args = dict(x=_apart(x, 24) if pitches else x)
        if xt == "f16":
            w = _np(torch.from_numpy(w).to(torch.float32).to(torch.float16))
    b = torch.randn(E, n, generator=gen, device="cuda").to(DT[out_t]) if bias else None
    out = torch.full((M, N), 9.0, dtype=DT[out_t], device="cuda")
    if pitches:
        big = torch.full((M, N + 7), 9.0, dtype=DT[out_t], device="cuda")
        out = big[:, 5:5 + N]
        q, s = _apart(q, 48), _apart(s, 3, 1)
    if E == 1 and not pitches:
        q, s = q[0], s[0]
    m.moe_mx_linear(w=q, w_scale=s, out=out, offsets=torch.from_numpy(off).cuda() if offsets else None, bias=b,
                    act=getattr(m, "ACT_" + act.upper()), stream=stream, **args)
    torch.cuda.synchronize()
    got, want = _np(out), OM.linear(xr, w, off, _np(b), act, np.full((M, N), 9.0))
    half = torch.finfo(DT[out_t]).eps / 2
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        bb = None if b is None else _np(b[e])
        z = OL.product(xr[lo:hi], w[e], bb)
        _, ey = _forward_error(xr[lo:hi], w[e], bb, act, z)
        y = want[lo:hi]
        bound = ey * (1 + half) + half * np.abs(y) + (2.0 ** -25 if out_t == "f16" else 0)
        err = np.abs(got[lo:hi] - y)
        assert np.all(err <= bound), (e, (err - bound).max(), np.argwhere(err > bound)[:4].tolist())
    assert np.all(got[~held] == 9)
    if pitches:
        assert bool((big[:, :5] == 9).all()) and bool((big[:, 5 + N:] == 9).all())
    return out


def _apart(t, more, at=0):
    """The same values in rows `more` elements further apart, from column `at` on, 255 (or NaN) between."""
    fill = 255 if t.dtype is torch.uint8 else float("nan")
    big = torch.full((*t.shape[:-1], t.shape[-1] + more), fill, dtype=t.dtype, device="cuda")
    big[..., at:at + t.shape[-1]] = t
    return big[..., at:at + t.shape[-1]]


TYPES = [("bf16", "bf16"), ("f16", "f32"), ("mx", "bf16")]
SIZES = [(1, 1, 32, 1), (1, 64, 2048, 1), (1, 200, 7168, 3), (2, 17, 64, 2), (5, 40, 96, 8), (8, 130, 1024, 64), (16, 48, 256, 1),
         (17, 100, 160, 4), (33, 36, 544, 2), (64, 96, 512, 128), (100, 250, 288, 5), (300, 130, 1056, 7), (700, 70, 128, 130),
         (513, 300, 224, 1), (1000, 260, 544, 3), (600, 300, 2336, 1), (200, 200, 2848, 2), (1300, 390, 1056, 2),
         (5000, 130, 96, 6)]


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("M,N,K,E", SIZES)
def test_product(M, N, K, E, act):
    for i, (xt, out_t) in enumerate(TYPES):
        _check(M, N, K, E, act, xt, out_t, kind=["even", "loud", "few"][(i + M) % 3], bias=(i + M) % 2 == 0)


# sizes that between them take every way of cutting a product, with sums over several tables of scales
CUTS = [(25, 2060, 1184, 8), (700, 130, 1184, 1), (601, 130, 672, 2), (97, 700, 1184, 32), (2001, 30, 1184, 2), (193, 390, 672, 64),
        (2500, 30, 2336, 1), (1281, 390, 1184, 64), (6401, 130, 672, 32), (22401, 30, 672, 32), (64001, 30, 672, 16), (9601, 130, 672, 64),
        (40001, 30, 1184, 16), (32001, 130, 672, 32), (22401, 130, 1184, 32), (2561, 700, 672, 64), (32001, 130, 1184, 64),
        (1601, 700, 1184, 64), (1600, 1030, 672, 64)]


def _values64(q, s):
    """What packed rows stand for, in float64 on the GPU (powers of two from a table: exact)."""
    power = torch.from_numpy(np.ldexp(1.0, np.arange(256) - 127)).cuda()[s.long()]
    return torch.from_numpy(OM.ELEMENTS).cuda()[torch.stack([q & 15, q >> 4], -1).flatten(-2).long()] * power.repeat_interleave(32, -1)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("M,N,K,E", CUTS)
def test_every_cut(M, N, K, E, act):
    """The same bound, with the float64 sums taken on the GPU: sizes too long for the oracle."""
    m = _m()
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    n = 2 * N if act == "swiglu" else N
    off = _offsets(M, E, "loud" if M % 2 else "even", np.random.default_rng(M))
    q, s = _weights(E, n, K, gen)
    x = torch.randn(M, K, generator=gen, device="cuda")
    b = torch.randn(E, n, generator=gen, device="cuda")
    for xt in ("bf16", "f16", "mx"):
        say(f"[mx linear] {M}x{N}x{K} E={E} {act} {xt}")
        out = torch.full((M, N), 9.0, device="cuda")
        if xt == "mx":
            xq, xs = _quantize(x)
            args, xr = dict(x=xq, x_scale=xs), _values64(xq, xs)
        else:
            args = dict(x=x.to(DT[xt]))
            xr = args["x"].double()
        # (fp16 holds these weights exactly: scales of 2^-9 to 2^-6)
        m.moe_mx_linear(w=q, w_scale=s, out=out, offsets=torch.from_numpy(off).cuda(), bias=b, act=getattr(m, "ACT_" + act.upper()), **args)
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            if lo == hi:
                continue
            w = _values64(q[e], s[e])
            z = torch.mm(xr[lo:hi], w.t().contiguous()) + b[e].double()
            ez = (K + 2) * U * (torch.mm(xr[lo:hi].abs(), w.t().contiguous().abs()) + b[e].double().abs())
            if act == "swiglu":
                g, u = z[:, :N], z[:, N:]
                y = g * torch.sigmoid(g) * u
                sg = (g * torch.sigmoid(g)).abs()
                ez = (1.13 * ez[:, :N] * u.abs() + sg * ez[:, N:] + 1.13 * ez[:, :N] * ez[:, N:] +
                      (16 * U + 64 * U * g.abs()) * sg * u.abs())
            else:
                y = z
            err = (out[lo:hi].double() - y).abs()
            assert bool((err <= ez * (1 + U) + U * y.abs()).all()), (xt, e, float((err - ez).max()))


@pytest.mark.parametrize("kind", ["even", "loud", "few", "ends"])
@pytest.mark.parametrize("xt", ["bf16", "f16", "mx"])
def test_ragged_experts(kind, xt):
    for M, N, K, E in ((37, 30, 160, 9), (400, 150, 320, 6), (1500, 90, 192, 70)):
        _check(M, N, K, E, "swiglu", xt, "f32", kind=kind)
        _check(M, N, K, E, "none", xt, "f32" if xt == "mx" else xt, kind=kind, bias=True)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
def test_activations_types_and_bias(act):
    for M, N, K, E in ((6, 44, 96, 2), (300, 140, 160, 2)):
        for xt, outs in (("bf16", ("bf16", "f32")), ("f16", ("f16", "f32")), ("mx", ("bf16", "f16", "f32"))):
            for out_t in outs:
                for bias in (False, True):
                    _check(M, N, K, E, act, xt, out_t, bias=bias)


@pytest.mark.parametrize("M,N,K,E", [(5, 33, 96, 3), (260, 150, 544, 3), (600, 300, 352, 2)])
@pytest.mark.parametrize("xt", ["bf16", "f16", "mx"])
def test_pitches(M, N, K, E, xt):
    for act in ("none", "swiglu"):
        _check(M, N, K, E, act, xt, "f32", kind="loud", pitches=True, bias=True)


@pytest.mark.parametrize("xt", ["bf16", "mx"])
def test_scales_over_a_wide_range(xt):
    for M, N, K in ((4, 40, 256), (300, 140, 512)):
        _check(M, N, K, 2, "none", xt, "f32", spread=30)


@pytest.mark.parametrize("M", [6, 300])
@pytest.mark.parametrize("xt", ["bf16", "f16", "mx"])
def test_scales_at_both_ends(M, xt):
    """One element a row of w, of every code over scales from 2^-127 to 2^127, times rows of a power of two each: every
    sum is one product, exact but for the ends of the types."""
    m = _m()
    K = 128
    scales = [0, 1, 2, 60, 101, 103, 112, 127, 141, 142, 190, 252, 253, 254]
    rows = [(c, s) for s in scales for c in range(1, 16) if c != 8]
    q, s = np.zeros((len(rows), K // 2), np.uint8), np.full((len(rows), K // 32), 254, np.uint8)
    for n, (c, sc) in enumerate(rows):
        at = (37 * n) % K
        q[n, at // 2] = c << (at % 2 * 4)
        s[n, at // 32] = sc
    w = OM.values(q, s)
    low, high = {"bf16": (-133, 127), "f16": (-24, 15), "mx": (-127, 127)}[xt]
    power = np.linspace(low, high, M).astype(np.int64)
    out = torch.empty(M, len(rows), device="cuda")
    qg, sg = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    if xt == "mx":
        x = torch.full((M, K // 2), 0x22, dtype=torch.uint8, device="cuda")           # 1 and 1
        xs = torch.from_numpy(np.repeat((power + 127).astype(np.uint8)[:, None], K // 32, 1)).cuda()
        m.moe_mx_linear(x, qg, sg, out, x_scale=xs)
    else:
        x = torch.from_numpy(np.repeat(np.ldexp(1.0, power)[:, None], K, 1)).to(DT[xt]).cuda()
        m.moe_mx_linear(x, qg, sg, out)
        w = _np(torch.from_numpy(w).float().to(DT[xt]))
    w = w.sum(1)                                       # the row's element (the others are zeros)
    with np.errstate(over="ignore"):
        want = (np.ldexp(1.0, power)[:, None] * w[None]).astype(np.float32)
    got = out.cpu().numpy()
    assert np.array_equal(got, want), [(int(power[i]), rows[j], got[i, j], want[i, j]) for i, j in np.argwhere(got != want)[:6]]


@pytest.mark.skipif(not (hasattr(torch, "float4_e2m1fn_x2") and hasattr(torch, "float8_e8m0fnu")), reason="no such types")
def test_bytes_under_their_own_types():
    m = _m()
    x = torch.randn(40, 128, device="cuda").bfloat16()
    q, s = _quantize(x)
    q4, s8 = q.view(torch.float4_e2m1fn_x2), s.view(torch.float8_e8m0fnu)
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    m.moe_mx_quantize(x, q2.view(torch.float4_e2m1fn_x2), s2.view(torch.float8_e8m0fnu))
    assert torch.equal(q, q2) and torch.equal(s, s2)
    back, back2 = torch.empty_like(x), torch.empty_like(x)
    m.moe_mx_dequantize(q, s, back)
    m.moe_mx_dequantize(q4, s8, back2)
    assert torch.equal(back, back2)
    y, y2 = torch.empty(40, 40, device="cuda"), torch.empty(40, 40, device="cuda")
    m.moe_mx_linear(q, q, s, y, x_scale=s)
    m.moe_mx_linear(q4, q4[None], s8[None], y2, x_scale=s8)
    assert torch.equal(y, y2)


def test_one_expert_without_offsets():
    for xt, out_t in TYPES:
        _check(40, 50, 96, 1, "none", xt, out_t, offsets=False)
        _check(300, 200, 160, 1, "swiglu", xt, out_t, offsets=False, pitches=True)


@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("xt", ["bf16", "f16", "mx"])
def test_what_is_not_a_number_stays_in_its_row_and_column(M, xt):
    m = _m()
    N, K = 150, 192
    gen = torch.Generator(device="cuda").manual_seed(M)
    q, s = _weights(1, N, K, gen)
    q, s = q[0], s[0]
    x = torch.randn(M, K, generator=gen, device="cuda")

    def run(x):
        out = torch.empty(M, N, device="cuda")
        if xt == "mx":
            xq, xs = _quantize(x)
            m.moe_mx_linear(xq, q, s, out, x_scale=xs)
        else:
            m.moe_mx_linear(x.to(DT[xt]), q, s, out)
        return out

    clean = run(x)
    x[1, 77] = float("nan")
    s[N - 2, 3] = 255
    out = run(x)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1] = True
    bad[:, N - 2] = True
    assert torch.equal(torch.isnan(out), bad) and torch.equal(out[~bad], clean[~bad])


def test_offsets_out_of_order_or_range_stay_inside_the_buffers():
    m = _m()
    for M in (20, 700):
        for xt in ("bf16", "mx"):
            big = torch.full((M + 8, 64), 9.0, device="cuda")
            q, s = _weights(4, 64, 64, torch.Generator(device="cuda").manual_seed(0))
            x = torch.randn(M, 64, device="cuda")
            xq, xs = _quantize(x)
            args = dict(x=xq, x_scale=xs) if xt == "mx" else dict(x=x.bfloat16())
            for off in ([-5, 3, 2, 2 ** 31 - 1, 10], [M + 4, 2, -2 ** 31, 5, 3 * M], [0, 0, 0, 0, 0]):
                m.moe_mx_linear(w=q, w_scale=s, out=big[4:4 + M], offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), **args)
                torch.cuda.synchronize()
                assert bool((big[:4] == 9).all()) and bool((big[4 + M:] == 9).all())
            assert bool((big == 9).sum() >= 8 * 64)


@pytest.mark.parametrize("M", [20, 700])
@pytest.mark.parametrize("xt", ["bf16", "f16", "mx"])
def test_rows_outside_every_experts_stay_as_they_were(M, xt):
    """Also with offsets out of order or range: what no expert's offsets, cut to the buffer, enclose is not written."""
    m = _m()
    q, s = _weights(4, 64, 64, torch.Generator(device="cuda").manual_seed(0))
    x = torch.randn(M, 64, device="cuda")
    if xt == "mx":
        xq, xs = _quantize(x)
        args = dict(x=xq, x_scale=xs)
    else:
        args = dict(x=x.to(DT[xt]))
    for off in ([0, 0, 0, 0, 0], [M, M, M, M, M], [M - 1, M - 1, M, M, M], [3, 3, M // 2, M // 2, M - 2], [0, 1, 1, 2, 2],
                [-5, 3, 2, 2 ** 31 - 1, 10], [M + 4, 2, -2 ** 31, 5, 3 * M], [9, 7, 5, 3, 1]):
        big = torch.full((M + 8, 64), 9.0, device="cuda")
        m.moe_mx_linear(w=q, w_scale=s, out=big[4:4 + M], offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), **args)
        touched = (big != 9).any(1).cpu().numpy()
        cut = np.clip(np.array(off, np.int64), 0, M)
        enclosed = np.zeros(M + 8, bool)
        for lo, hi in zip(cut, cut[1:]):
            enclosed[4 + lo:4 + max(hi, lo)] = True
        assert not (touched & ~enclosed).any(), off
        if (np.diff(off) >= 0).all():
            assert np.array_equal(touched, enclosed), off       # (a result of 9 in all 64 columns aside)


def test_no_rows():
    m = _m()
    q, s = _weights(2, 64, 64, torch.Generator(device="cuda").manual_seed(0))
    m.moe_mx_linear(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), q, s, torch.empty(0, 64, device="cuda"),
                    offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
