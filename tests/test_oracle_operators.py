"""The oracle of the operators around the experts: closed forms and differences."""
import numpy as np
import pytest

from oracle import linear as OL
from oracle import route as OR


def test_route_by_hand():
    z = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = OR.route(z, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 0.25]])
    ids, w = OR.route(z, 3, renorm=True, scale=2.0)
    assert ids.tolist() == [[2, 1, 0]] and np.allclose(w, 2 * np.array([[4, 2, 1]]) / 7)   # tie: lower id
    ids, w = OR.route(z, 2, kind="sigmoid", bias=[0.0, 0.0, -1.0, 0.5])
    assert ids.tolist() == [[3, 1]] and np.allclose(w, [[0.5, 2 / 3]])
    # groups {0, 1} and {2, 3}: maxima 0.25 and 0.5; a dropped group's experts come last with weight 0
    ids, w = OR.route(z, 2, n_group=2, topk_group=1)
    assert ids.tolist() == [[2, 3]]
    z[0, 2:] = -np.inf
    ids, w = OR.route(z, 4)
    assert ids.tolist() == [[1, 0, 2, 3]] and np.allclose(w, [[2 / 3, 1 / 3, 0, 0]])
    ids, w = OR.route(np.full((1, 3), -np.inf), 2, renorm=True)
    assert ids.tolist() == [[0, 1]] and not w.any()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_difference_quotient(kind, renorm):
    rng = np.random.default_rng(3)
    z = rng.standard_normal((4, 7))
    ids, w = OR.route(z, 3, kind=kind, renorm=renorm, scale=1.5)
    held = w != 0
    held[1, 2] = False
    g = rng.standard_normal((4, 3))
    got = OR.route_backward(z, ids, held, g, kind=kind, renorm=renorm, scale=1.5)
    h = 1e-6
    for t in range(4):
        for e in range(7):
            d = np.zeros_like(z)
            d[t, e] = h
            f = [(g * OR.weights_of(z + s * d, ids, held, kind, renorm, 1.5)).sum() for s in (1, -1)]
            assert abs((f[0] - f[1]) / (2 * h) - got[t, e]) < 1e-8


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
def test_linear_gradient_is_the_difference_quotient(act):
    rng = np.random.default_rng(5)
    n = 6 if act == "swiglu" else 3
    x, w, b = rng.standard_normal((4, 5)), rng.standard_normal((n, 5)), rng.standard_normal(n)
    g = rng.standard_normal((4, 3))
    pre = OL.product(x, w, b)
    d = OL.dz(act, g, pre)

    def loss(x, w, b):
        return (g * OL.apply(act, OL.product(x, w, b))).sum()

    h = 1e-6
    for arr, grad in ((x, d @ w), (w, d.T @ x), (b, d.sum(0))):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = loss(x, w, b)
            arr[i] = keep - h
            down = loss(x, w, b)
            arr[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7
