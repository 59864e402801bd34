"""The dense operators' oracle against closed forms, finite differences and brute force (CPU)."""
import math

import numpy as np
import pytest

from oracle import dense


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_act_grad_matches_differences(name):
    v = np.linspace(-6, 6, 101)
    h = 1e-6
    num = (dense.act(v + h, name) - dense.act(v - h, name)) / (2 * h)
    # the central difference is off by h^2/6 |f'''| (below 1e-12) plus rounding, 2 * 2^-53 * 6 / h
    assert np.abs(num - dense.act_grad(v, name)).max() < 1e-8


def test_rmsnorm_of_constant_rows():
    x = np.array([[2.0] * 8, [0.0] * 8])
    v, y = dense.rmsnorm(x, None, np.arange(8.0), 0.0 + 1e-30)
    assert np.allclose(y[0], np.arange(8.0)) and np.all(y[1] == 0) and np.array_equal(v, x)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_backward_matches_differences(act):
    rng = np.random.default_rng(0)
    T, H, I = 3, 4, 5
    x, w13, w2 = rng.standard_normal((T, H)), rng.standard_normal((2 * I, H)), rng.standard_normal((H, I))
    dy = rng.standard_normal((T, H))

    def loss(x, w13, w2):
        return float((dense.glu(x, w13, act)[2] @ w2.T * dy).sum())

    g, u, _ = dense.glu(x, w13, act)
    grads = dense.ffn_backward(dy, x, g, u, w13, w2, act)
    h = 1e-5
    for which, grad in enumerate(grads):
        args = [x, w13, w2]
        for at in np.ndindex(*grad.shape):
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[which][at] += h
            dn[which][at] -= h
            # third derivatives of order 100 times h^2 / 6, plus rounding 1e-15 * 100 / h
            assert abs((loss(*up) - loss(*dn)) / (2 * h) - grad[at]) < 1e-6


def test_route_special_rows():
    inf = math.inf
    lg = np.array([[1, 3, 3, 2], [-inf, math.nan, 0, -inf], [-inf] * 4, [inf, 0, inf, 1]], np.float32)
    ids, w = dense.route(lg, 2, "softmax", True, 1.0)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [0, 2]]
    assert np.allclose(w, [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5]])
