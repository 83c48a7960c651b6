"""Orders that 32 bits do not decide: rows built so that the ranking of
c = score + bias hangs on the error of a 32-bit score, against the float64
oracle.  Ids have to be equal."""
import numpy as np
import pytest
import torch

from gpu_helpers import say
from oracle import route as OR

pytestmark = pytest.mark.gpu


def _ids(z, k, kind, bias, **kw):
    import moe_expert_tile_amd as m
    T = z.shape[0]
    zd = torch.from_numpy(z).cuda()
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    m.moe_route(zd, ids, w, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                score=m.SCORE_SIGMOID if kind == "sigmoid" else m.SCORE_SOFTMAX, n_group=kw.get("n_group", 1),
                topk_group=kw.get("topk_group", 0), group_score=m.GROUP_TOP2 if kw.get("top2") else m.GROUP_MAX)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy()


def _bias_for(c, s):
    """fp32 biases that bring scores s to about c."""
    return (np.asarray(c, np.float64) - s).astype(np.float32)


@pytest.mark.parametrize("E", [24, 100, 256, 512, 1024])
def test_a_large_score_below_the_first_one_left_out(E):
    """Expert 0 holds nearly all of the softmax under a bias of about -0.99,
    so its c is off by many times the other experts' error.  Experts 8 and 9
    come after it by 1e-7 and 4.6e-7: 32 bits may rank it behind both, and 8
    and 9 are not close by their own errors."""
    z = np.full((1, E), -16.6, np.float32)
    z[0, 0] = 0.0
    s = OR.scores(z, "softmax")[0]
    c0 = s[0] + float(np.float32(-0.99))
    c = c0 - 0.002 - 1e-4 * np.arange(E)
    c[1:8] = c0 + 0.1 + 0.01 * np.arange(7)
    c[8], c[9] = c0 - 1e-7, c0 - 4.6e-7
    bias = _bias_for(c, s)
    bias[0] = np.float32(-0.99)
    ids, _ = _ids(z, 8, "softmax", bias)
    want, _ = OR.route(z, 8, kind="softmax", bias=bias)
    assert 0 in want[0] and np.array_equal(ids, want), (ids, want)


@pytest.mark.parametrize("E,k,seed", [(24, 4, 0), (100, 8, 1), (128, 3, 2), (256, 8, 3), (256, 30, 4), (512, 6, 5),
                                      (777, 9, 6), (1024, 8, 7)])
@pytest.mark.parametrize("groups", [1, 4])
def test_a_large_score_among_near_ones(E, k, seed, groups):
    """One large score with a negative bias moves through a ladder of experts
    a few 1e-7 apart as the other logits shift."""
    rng = np.random.default_rng(seed)
    if E % groups:
        groups = 1
    T = 96
    z = (rng.uniform(-17.5, -14.0, (T, 1)) + rng.uniform(-0.2, 0.2, (1, E))).astype(np.float32)
    big = int(rng.integers(E))
    z[:, big] = rng.uniform(-0.5, 0.5)
    s = OR.scores(z, "softmax")
    b0 = np.float32(-0.97)
    mid = float(np.median(s[:, big] + float(b0)))
    order = rng.permutation(E)
    c = np.empty(E)
    c[order] = mid + (k - np.arange(E)) * rng.uniform(1e-7, 6e-7, E) - 1e-3 * (np.arange(E) > 2 * k)
    bias = _bias_for(c, s.mean(0))
    bias[big] = b0
    for kw in ({}, dict(n_group=groups, topk_group=max(1, groups // 2)),
               dict(n_group=groups, topk_group=max(1, groups // 2), top2=True)):
        kk = min(k, E // groups) if kw else k
        say(f"[route order] E={E} k={kk} {kw}")
        ids, _ = _ids(z, kk, "softmax", bias, **kw)
        want, _ = OR.route(z, kk, kind="softmax", bias=bias, **kw)
        assert np.array_equal(ids, want), np.argwhere(ids != want)[:4]


def test_a_tie_in_front_of_a_near_one():
    """Experts 8 and 9 have the same logit and bias; expert 10 is above both
    by less than a 32-bit step.  With one pick the first one left out is 9,
    which the index decides, and 10 lies behind it."""
    step = 2.0 ** -22                       # of a 32-bit c between 2 and 4
    rng = np.random.default_rng(0)

    def member(offset):                     # (logit, bias): c at a step's middle + offset, to 1e-8
        while True:
            zz = rng.uniform(-1, 1, 1 << 20).astype(np.float32)
            s = 1 / (1 + np.exp(-zz.astype(np.float64)))
            b = (3.0 - s).astype(np.float32)
            c = s + b.astype(np.float64)
            hit = np.abs(c - (3.0 + offset)) < 1e-8
            if hit.any():
                return zz[hit][0], b[hit][0]

    low, high = member(-step / 6), member(step / 6)
    z, bias = np.zeros((3, 64), np.float32), np.zeros(64, np.float32)
    z[:, 8:10], bias[8:10] = low[0], low[1]
    z[:, 10], bias[10] = high
    for k in (1, 2, 3):
        ids, _ = _ids(z, k, "sigmoid", bias)
        want, _ = OR.route(z, k, kind="sigmoid", bias=bias)
        assert want[0, 0] == 10 and np.array_equal(ids, want), (k, ids)


@pytest.mark.parametrize("E,k", [(64, 1), (256, 8), (1024, 30)])
def test_ties_around_the_last_pick(E, k):
    """16-bit logits and equal biases: the k-th pick and many left out are the
    same expert but for the index."""
    rng = np.random.default_rng(E)
    z = np.round(rng.standard_normal((200, E)) * 2) / 2
    z = z.astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        for bias in (np.zeros(E, np.float32), np.where(np.arange(E) % 3, 0.25, 0.125).astype(np.float32)):
            ids, _ = _ids(z, k, kind, bias)
            want, _ = OR.route(z, k, kind=kind, bias=bias)
            assert np.array_equal(ids, want)


@pytest.mark.parametrize("E,G", [(16, 4), (64, 8), (256, 8), (1024, 64)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_a_group_of_one_expert_with_an_infinite_bias(E, G, kind):
    """A +inf bias puts its expert first.  Its group's two best are +inf and a
    masked expert, so under the sum of two the group ranks as masked; under
    the maximum, or with a second expert, it ranks first."""
    size = E // G
    rng = np.random.default_rng(E)
    z = rng.standard_normal((20, E)).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    bias[E - 1] = np.inf
    alone = z.copy()
    alone[:, E - size:E - 1] = -np.inf
    for logits, top2 in ((alone, True), (alone, False), (z, True), (z, False)):
        for k in (1, 3):
            kw = dict(n_group=G, topk_group=2, top2=top2)
            ids, w = _ids(logits, k, kind, bias, **kw)
            want, ww = OR.route(logits, k, kind=kind, bias=bias, **kw)
            assert np.array_equal(ids, want), (ids[:3], want[:3])
            assert np.all(np.abs(w - ww) <= 2.0 ** -18 * ww)
            assert (ids[:, 0] == E - 1).all() == (not (top2 and logits is alone))


def test_several_infinite_biases():
    """+inf ones rank first among themselves by index, then the others; near
    ones behind them are still ranked in 64 bits."""
    rng = np.random.default_rng(3)
    z = np.repeat(rng.standard_normal((1, 96)), 30, 0).astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        bias = _bias_for(np.full(96, 0.5), OR.scores(z[:1], kind)[0])
        bias[[70, 11, 40]] = np.inf
        bias[5] = -np.inf
        for k in (1, 2, 3, 4, 12):
            for kw in ({}, dict(n_group=8, topk_group=4), dict(n_group=8, topk_group=4, top2=True)):
                ids, _ = _ids(z, k, kind, bias, **kw)
                want, _ = OR.route(z, k, kind=kind, bias=bias, **kw)
                assert np.array_equal(ids, want), (k, kw)
