"""Routing and its gradient on the GPU against the float64 oracle.

Ids have to be equal (the oracle ranks in 64 bits).  Tolerances, for values
held in 32 bits with u = 2^-24 (half a step): a weight's exponent z - max has
an error of u |z - max| (below 32 u here), exp, division and products a few u,
a sum over E <= 1024 experts at most (16 + 10) u in its order of summation:
below 64 u = 2^-18 relative.  A gradient is a sum of products of such weights
and the given g: 2^-17 of scale max|g| on top of its own rounding to the
logits' type.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import route as OR

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _m():
    import moe_expert_tile_amd as m
    return m


def _call(z, k, kind="softmax", bias=None, renorm=False, n_group=1, topk_group=0, top2=False, scale=1.0):
    m = _m()
    ids = torch.full((z.shape[0], k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((z.shape[0], k), -7.0, device="cuda")
    m.moe_route(z, ids, w, bias=bias, score=m.SCORE_SIGMOID if kind == "sigmoid" else m.SCORE_SOFTMAX, renorm=renorm,
                n_group=n_group, topk_group=topk_group, group_score=m.GROUP_TOP2 if top2 else m.GROUP_MAX,
                scale=scale)
    torch.cuda.synchronize()
    return ids, w


def _check(z, k, **kw):
    ids, w = _call(z, k, **kw)
    host = dict(kw, bias=None if kw.get("bias") is None else kw["bias"].double().cpu().numpy())
    rid, rw = OR.route(z.double().cpu().numpy(), k, **host)
    assert np.array_equal(ids.cpu().numpy(), rid)
    err = np.abs(w.double().cpu().numpy() - rw)
    # absolute term: weights below fp32's smallest normal number flush
    assert np.all(err <= 2.0 ** -18 * np.abs(rw) + 2.0 ** -125), err.max()
    return ids, w


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (3, 5, 5), (64, 8, 2), (65, 16, 9), (7, 17, 3), (257, 60, 6),
                                   (64, 64, 32), (33, 100, 8), (130, 128, 8), (5, 160, 10), (1, 256, 8), (66, 256, 32),
                                   (40, 257, 4), (9, 384, 8), (17, 512, 1), (6, 777, 20), (12, 1024, 8),
                                   (3, 1024, 32)])
def test_topk(T, E, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T * 1000 + E)
    z = (torch.randn(T, E, generator=gen, device="cuda") * 2).to(DT[dtype])
    bias = torch.randn(E, generator=gen, device="cuda") * 0.2
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            say(f"[route] T={T} E={E} k={k} {dtype} {kind} renorm={renorm}")
            _check(z, k, kind=kind, renorm=renorm, scale=1.0)
            _check(z, k, kind=kind, renorm=renorm, bias=bias, scale=2.5)


@pytest.mark.parametrize("E,G,keep,k", [(8, 8, 3, 3), (16, 4, 1, 4), (15, 3, 2, 5), (60, 6, 2, 6), (64, 8, 3, 8),
                                        (160, 8, 3, 6), (256, 8, 4, 8), (256, 16, 5, 30), (256, 1, 1, 8),
                                        (96, 32, 7, 9), (1023, 33, 4, 12), (1024, 64, 9, 32), (1020, 5, 2, 7),
                                        (340, 17, 3, 8), (12, 2, 2, 12)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_groups(E, G, keep, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(E + G)
    z = (torch.randn(37, E, generator=gen, device="cuda") * 2).to(DT[dtype])
    bias = torch.randn(E, generator=gen, device="cuda") * 0.2
    for top2 in (False, True):
        if top2 and E // G < 2:
            continue
        for b in (None, bias):
            for kind in ("softmax", "sigmoid"):
                say(f"[groups] E={E} G={G} keep={keep} k={k} {dtype} top2={top2} bias={b is not None} {kind}")
                _check(z, k, kind=kind, renorm=True, bias=b, n_group=G, topk_group=keep, top2=top2, scale=2.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_masked_experts_and_empty_rows(dtype, kind):
    """-inf logits, whole rows of them, the type's lowest value and dead experts by their bias."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(50, 40, generator=gen, device="cuda").to(DT[dtype])
    z[torch.rand(50, 40, generator=gen, device="cuda") < 0.8] = -float("inf")
    z[3] = -float("inf")
    z[4] = torch.finfo(DT[dtype]).min
    z[5, ::2] = torch.finfo(DT[dtype]).min
    bias = torch.randn(40, generator=gen, device="cuda") * 0.1
    bias[7] = -float("inf")
    for renorm in (False, True):
        for b in (None, bias):
            ids, w = _check(z, 8, kind=kind, renorm=renorm, bias=b)
            assert ids[3].tolist() == list(range(8)) and not w[3].any()
            if b is not None:
                assert not w[ids == 7].any()
            _check(z, 6, kind=kind, renorm=renorm, bias=b, n_group=8, topk_group=3, top2=True)
            _check(z, 6, kind=kind, renorm=renorm, bias=b, n_group=8, topk_group=3)


def test_ties_go_to_the_lower_expert():
    z = torch.zeros(5, 256, device="cuda", dtype=torch.bfloat16)
    z[1, 100:] = 1.0
    z[2] = -0.0
    z[2, 9] = 0.0
    z[3] = torch.arange(256, device="cuda") // 32
    z[4] = (torch.arange(256, device="cuda") % 3).flip(0)
    for kw in (dict(), dict(bias=torch.zeros(256, device="cuda")), dict(bias=torch.full((256,), 3.0, device="cuda")),
               dict(n_group=8, topk_group=2), dict(n_group=8, topk_group=2, top2=True)):
        for kind in ("softmax", "sigmoid"):
            _check(z, 8, kind=kind, **kw)


def test_near_ties_are_ranked_in_64_bits():
    """Scores plus biases that agree in 32 bits and differ beyond: a shifted
    bias undoes the logits' differences up to 2^-40."""
    rng = np.random.default_rng(2)
    T, E = 64, 48
    z = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    z[:] = z[0]
    for kind in ("softmax", "sigmoid"):
        s = OR.scores(z[:1].double().cpu().numpy(), kind)[0]
        bias = torch.from_numpy((0.5 - s).astype(np.float32)).cuda()   # c = 0.5 + rounding errors of 2^-26
        _check(z, 10, kind=kind, renorm=True, bias=bias)
        _check(z, 10, kind=kind, renorm=True, bias=bias, n_group=6, topk_group=3, top2=True)
        _check(z, 10, kind=kind, renorm=True, bias=bias, n_group=6, topk_group=3)
        _check(z, 32, kind=kind, renorm=True, bias=bias + 1000.0)


def test_saturated_and_far_scores():
    z = torch.tensor([[30.0, 29.0, -20.0, 25.0, -60.0, 28.0, 0.0, 27.5],
                      [-200.0, -201.0, -199.5, -210.0, -250.0, -260.0, -198.0, -1000.0],
                      [80.0, -80.0, 79.0, -79.0, 1.0, 2.0, 3.0, 4.0]], device="cuda")
    for k in (1, 3, 8):
        _check(z, k, kind="sigmoid")
        _check(z, k, kind="softmax")
        _check(z, k, kind="softmax", renorm=True)
    # weights of far negative logits keep their ratios
    ids, w = _call(z[1:2], 3, kind="sigmoid", renorm=True)
    e = np.exp(np.array([0.0, -1.5, -2.0]))
    assert ids.tolist() == [[6, 2, 0]] and np.allclose(w.cpu().numpy()[0], e / e.sum(), rtol=2.0 ** -18)


def test_nan_rows_and_infinities():
    z = torch.randn(6, 64, device="cuda")
    z[1, 5] = float("nan")
    z[2, 6] = float("inf")
    z[3] = float("nan")
    for kw in (dict(), dict(bias=torch.zeros(64, device="cuda")), dict(n_group=4, topk_group=2, top2=True)):
        for kind in ("softmax", "sigmoid"):
            ids, w = _call(z, 8, kind=kind, **kw)
            for t in range(6):
                assert len(set(ids[t].tolist())) == 8 and min(ids[t].tolist()) >= 0 and max(ids[t].tolist()) < 64
            bad = [False, True, kind == "softmax", True, False, False]
            assert torch.isnan(w).all(1).tolist() == bad and torch.isnan(w).any(1).tolist() == bad
    bias = torch.zeros(64, device="cuda")
    bias[3] = float("nan")
    _, w = _call(z[4:], 8, bias=bias)
    assert torch.isnan(w).all()


def test_strides_and_unaligned_views():
    base = torch.randn(70, 203, device="cuda")
    base[:, :3] = float("nan")
    base[:, 163:] = float("inf")
    for dtype in DT.values():
        z = base.to(dtype)[:, 3:163]
        _check(z, 8, renorm=True)
        _check(z, 8, renorm=True, kind="sigmoid", bias=torch.randn(160, device="cuda"), n_group=8, topk_group=3, top2=True)
    wide = torch.randn(9, 320, device="cuda")
    _check(wide[:, 64:128], 8)
    _check(wide[::2, 64:128], 8)
    _check(wide.to(torch.bfloat16)[:, 64:128], 8)


def test_no_tokens():
    _call(torch.empty(0, 16, device="cuda"), 2)


# --- gradient ------------------------------------------------------------------

def _check_back(z, ids, w, g, kind, renorm, scale):
    m = _m()
    dz = torch.full_like(z, 7.0)
    m.moe_route_backward(z, ids, w, g, dz, score=m.SCORE_SIGMOID if kind == "sigmoid" else m.SCORE_SOFTMAX,
                         renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    held = (w != 0).cpu().numpy()
    ref = OR.route_backward(z.double().cpu().numpy(), ids.cpu().numpy(), held, g.double().cpu().numpy(), kind=kind,
                            renorm=renorm, scale=scale)
    err = np.abs(dz.double().cpu().numpy() - ref)
    half = torch.finfo(z.dtype).eps / 2
    # fp16's smallest step below its normal range
    tiny = 2.0 ** -25 if z.dtype is torch.float16 else 0.0
    assert np.all(err <= half * np.abs(ref) + 2.0 ** -17 * scale * float(g.abs().max()) + tiny), err.max()
    return dz


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (2, 5, 2), (65, 8, 2), (33, 60, 6), (9, 127, 8), (70, 256, 8), (5, 256, 32),
                                   (3, 777, 9), (4, 1024, 8), (2, 1024, 32)])
def test_gradient(T, E, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T * 7 + E)
    z = (torch.randn(T, E, generator=gen, device="cuda") * 2).to(DT[dtype])
    g = torch.randn(T, k, generator=gen, device="cuda")
    bias = torch.randn(E, generator=gen, device="cuda") * 0.2
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            say(f"[route back] T={T} E={E} k={k} {dtype} {kind} renorm={renorm}")
            ids, w = _call(z, k, kind=kind, renorm=renorm, bias=bias, scale=1.5)
            _check_back(z, ids, w, g, kind, renorm, 1.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_masked_strided_and_listed_twice(kind, renorm):
    gen = torch.Generator(device="cuda").manual_seed(11)
    z = torch.randn(40, 67, generator=gen, device="cuda")
    z[torch.rand(40, 67, generator=gen, device="cuda") < 0.9] = -float("inf")
    z[3] = -float("inf")
    g = torch.randn(40, 6, generator=gen, device="cuda")
    view = torch.full((40, 80), float("nan"), device="cuda")[:, 5:72]
    view.copy_(z)
    ids, w = _call(view, 6, kind=kind, renorm=renorm)
    dz = _check_back(view, ids, w, g, kind, renorm, 1.0)
    assert not dz[3].any() and torch.isfinite(dz).all()
    # the same expert in several slots: their contributions add up
    z = torch.randn(16, 24, generator=gen, device="cuda")
    ids = torch.randint(0, 24, (16, 6), generator=gen, device="cuda", dtype=torch.int32)
    ids[:, 3] = ids[:, 1]
    ids[:4] = ids[:4, :1]
    held = np.ones((16, 6), bool)
    w = torch.from_numpy(OR.weights_of(z.double().cpu().numpy(), ids.cpu().numpy(), held, kind, renorm)).float().cuda()
    _check_back(z, ids.contiguous(), w, g[:16].contiguous(), kind, renorm, 1.0)


def test_gradient_ignores_ids_out_of_range():
    m = _m()
    z, g = torch.randn(8, 16, device="cuda"), torch.randn(8, 4, device="cuda")
    ids, w = _call(z, 4)
    bad = ids.clone()
    bad[:, 2] = torch.tensor([-1, 16, 2 ** 30, -2 ** 31, 17, -5, 100, 16], device="cuda")
    bad[0] = -1
    a, b = torch.empty_like(z), torch.empty_like(z)
    m.moe_route_backward(z, bad, w, g, a)
    w0 = w.clone()
    w0[:, 2] = 0
    w0[0] = 0
    m.moe_route_backward(z, ids, w0, g, b)
    assert torch.equal(a, b) and not a[0].any()


def test_gradient_of_a_nan_row_stays_in_it():
    m = _m()
    z, g = torch.randn(8, 16, device="cuda"), torch.randn(8, 4, device="cuda")
    z[2, 3] = float("nan")
    ids, w = _call(z, 4)
    d = torch.empty_like(z)
    m.moe_route_backward(z, ids, w, g, d)
    assert torch.isnan(d).any(1).tolist() == [i == 2 for i in range(8)]


def test_offsets_beyond_32_bits():
    """2^23 + 5 tokens over 264 experts are 2.2e9 logits: the last tokens as in a small call."""
    m = _m()
    T, E, k = (1 << 23) + 5, 264, 4
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    z[-300:] = torch.randn(300, E, device="cuda").to(torch.bfloat16)
    say("[route] 2^23 tokens")
    ids, w = _call(z, k, kind="softmax")
    few, fw = _call(z[-300:].contiguous(), k, kind="softmax")
    assert torch.equal(ids[-300:], few) and torch.equal(w[-300:], fw)
    assert ids[12345].tolist() == [0, 1, 2, 3]
    g = torch.randn(T, k, device="cuda")
    d, ds = torch.empty_like(z), torch.empty(300, E, dtype=torch.bfloat16, device="cuda")
    m.moe_route_backward(z, ids, w, g, d)
    m.moe_route_backward(z[-300:].contiguous(), few, fw, g[-300:].contiguous(), ds)
    torch.cuda.synchronize()
    assert torch.equal(d[-300:], ds)


def test_long_batches_of_middle_sizes():
    """65 to 128 experts and 16384 tokens on take other lanes than short batches:
    the same result, row by row, as in short calls (compared with the oracle above)."""
    for E, k, G in ((100, 8, 1), (128, 8, 4), (72, 12, 8), (127, 6, 1)):
        z = torch.randn(16400, E, device="cuda")
        bias = torch.randn(E, device="cuda") * 0.1
        for b in (None, bias):
            kw = dict(kind="sigmoid", bias=b, renorm=True, n_group=G, topk_group=max(1, G // 2), top2=G > 1)
            ids, w = _call(z, k, **kw)
            for t in (0, 5000, 16000):
                few, fw = _call(z[t:t + 400].contiguous(), k, **kw)
                assert torch.equal(ids[t:t + 400], few)
                assert bool(((w[t:t + 400] - fw).abs() <= 2.0 ** -18 * fw).all())
            _check(z[:40].contiguous(), k, **kw)


def test_default_options_through_the_c_entry_point():
    m = _m()
    z = torch.randn(20, 24, device="cuda")
    ids, w = torch.zeros(20, 3, dtype=torch.int32, device="cuda"), torch.zeros(20, 3, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert m._lib.moe_route(20, 24, 3, z.data_ptr(), 2, 0, None, None, ids.data_ptr(), w.data_ptr(), s) == m.MOE_OK
    want, ww = _check(z, 3)
    assert torch.equal(ids, want) and torch.equal(w, ww)
    d, dn, g = torch.empty_like(z), torch.empty_like(z), torch.randn(20, 3, device="cuda")
    assert m._lib.moe_route_backward(20, 24, 3, z.data_ptr(), 2, 0, ids.data_ptr(), w.data_ptr(), g.data_ptr(), None,
                                     d.data_ptr(), 0, s) == m.MOE_OK
    m.moe_route_backward(z, ids, w, g, dn)
    assert torch.equal(d, dn)
