"""The check of the gradients against differences can tell right ones from wrong ones (CPU): gradients rounded as the
library rounds them pass it everywhere, and each of the mistakes one could make in them does not."""
import numpy as np
import pytest

import gradient_bounds as gb
from oracle import dense

SIZES = [(5, 24, 16), (1, 16, 8)]


def _bf16(a):
    """numpy fp64 -> the nearest bf16 values (ties to even)."""
    b = np.asarray(a, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def _gradients(x, w13, w2, dy, act, slope=None, scale=(1.0, 1.0)):
    I = w2.shape[1]
    gu = _bf16(x @ w13.T)
    g, u = gu[:, :I], gu[:, I:]
    s = dense.act_grad(g, act) if slope is None else slope(g)
    dh, a = dy @ w2, dense.act(g, act)
    dgu = _bf16(np.concatenate([dh * u * s * scale[0], dh * a * scale[1]], 1))
    return _bf16(dgu @ w13), _bf16(dgu.T @ x), _bf16(dy.T @ _bf16(a * u))


def _sigmoid(v):
    return 1 / (1 + np.exp(-v))


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_right_and_wrong_gradients(T, H, I, act):
    p = gb.point(T, H, I, act, 7, _bf16)
    want, tol = gb.differences(*p, act), gb.bounds(*p, act)
    for g, w, t in zip(_gradients(*p, act), want, tol):
        assert (np.abs(g - w) <= t).all()
    gelu_cdf = lambda v: dense.act(v, "gelu") / v                              # noqa: E731
    # the term v p'(v) missing, no slope, the activation for its slope, one half or a tenth of everything missing
    wrong = [dict(slope=_sigmoid if act == "silu" else gelu_cdf),
             dict(slope=lambda v: np.ones_like(v)), dict(slope=lambda v: dense.act(v, act)),
             dict(scale=(0.0, 1.0)), dict(scale=(1.0, 0.0)), dict(scale=(0.9, 0.9))]
    for kw in wrong:
        got = _gradients(*p, act, **kw)
        for g, w, t in zip(got[:2], want[:2], tol[:2]):
            assert (np.abs(g - w) > t).mean() > 0.1, (kw, "passes")
    u = p[0] @ p[1][I:].T
    for h in (u, 0.9 * dense.glu(p[0], p[1], act)[2]):                        # dw2 of h without its gate, or 10% off
        assert (np.abs(p[3].T @ h - want[2]) > tol[2]).mean() > 0.3
