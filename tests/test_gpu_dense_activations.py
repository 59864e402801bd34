"""The activations and their slopes at exactly known arguments, through every kind of kernel that applies them
(MI355X only): products with a single nonzero term leave no error of a sum to hide behind, and the tolerances
are relative, so the tails count as much as the middle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import dense
from scipy import special
from test_gpu_dense import BF, DEV, _bf, _np, _within

pytestmark = pytest.mark.gpu
VALUES = np.linspace(-12, 12, 769)


def _cdf(v):
    return 0.5 * special.erfc(-v / np.sqrt(2.0))


def _act(v, act):
    return v * special.expit(v) if act == "silu" else v * _cdf(v)


def _slope(v, act):
    if act == "silu":
        p = special.expit(v)
        return p + v * p * (1 - p)
    return _cdf(v) + v * np.exp(-0.5 * v * v) / np.sqrt(2 * np.pi)


def _rel(v, act):
    """Relative error of the activation in fp32.

    GELU: the tail is exp(-v^2 / 2) times a fitted function of |v|.  The exponent is off by 3 roundings of v^2 / 2,
    1.5 v^2 2^-24; the exponential and a reciprocal by 2 units in the last place each; the function, nine terms whose
    magnitudes add up to 2.5 times their sum at most, by some 2 * 2.5 * 2^-24 * 2 and its fit; three products.  Together
    (1.5 v^2 + 26) 2^-24 at most.
    SiLU: the exponent's argument is off by 2^-23 |v| (constant and product), the exponential by 2 units more, then a
    sum, and a division."""
    return ((v * v + 18) if act == "gelu" else (np.abs(v) + 4)) * 2.0 ** -23


def _slope_err(v, act):
    if act == "gelu":
        # exp(-v^2 / 2): two products and a constant in an argument of that size, and 2 units
        pdf = np.abs(v) * np.exp(-0.5 * v * v) / np.sqrt(2 * np.pi)
        return _cdf(v) * _rel(v, act) + pdf * (v * v + 4) * 2.0 ** -23 + 2.0 ** -24 * (_cdf(v) + pdf)
    # p (1 + v (1 - p)): 1 - p is off by p's own error and a rounding, absolutely
    p = special.expit(v)
    e_p = _rel(v, act)
    return p * ((e_p * p + 2.0 ** -23) * np.abs(v) + (e_p + 2.0 ** -22) * (1 + np.abs(v) * (1 - p)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("few", [True, False])
def test_linear_activations(act, dt, few):
    """y[t, n] = act(x[t, 0] w[n, 0]): the values down the rows or, for the kernel of few rows, along the columns."""
    v, vv = _bf(VALUES)
    n = len(VALUES)
    one, many = torch.zeros((3, 8), dtype=torch.bfloat16, device=DEV), torch.zeros((n, 8), dtype=torch.bfloat16, device=DEV)
    one[:, 0], many[:, 0] = 1, v
    out = torch.zeros((3, n) if few else (n, 3), dtype=dt, device=DEV)
    pe.linear(one if few else many, many if few else one, out, act=act)
    torch.cuda.synchronize()
    y = _act(vv, act)
    rel = _rel(vv, act)
    tol = np.abs(y) * (rel + (BF * (1 + rel) if dt == torch.bfloat16 else 0.0))
    got = _np(out) if few else _np(out).T
    for r in got:
        _within(r, y, tol, act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [2, 40])
def test_glu_activations(act, T):
    """h = act(g) * u with g the values and u = 1."""
    v, vv = _bf(VALUES[:768])
    I = len(vv)
    x = torch.zeros((T, 8), dtype=torch.bfloat16, device=DEV)
    w13 = torch.zeros((2 * I, 8), dtype=torch.bfloat16, device=DEV)
    x[:, 0], w13[:I, 0], w13[I:, 0] = 1, v, 1
    out = torch.zeros((T, I), dtype=torch.bfloat16, device=DEV)
    pe.glu(x, w13, out, act=act)
    torch.cuda.synchronize()
    y, rel = _act(vv, act), _rel(vv, act)
    for r in _np(out):
        _within(r, y, np.abs(y) * (rel + BF * (1 + rel)), act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_of_activations(act):
    """dg = act'(g), du = act(g) and h = act(g), for dh = u = 1."""
    v, vv = _bf(VALUES[:768])
    T, H, I = 3, 8, len(vv)
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)           # noqa: E731
    dy, w2, gu, dgu, h, dw2 = e(T, H), e(H, I), e(T, 2 * I), e(T, 2 * I), e(T, I), e(H, I)
    dy[:, 0], w2[0], gu[:, :I], gu[:, I:] = 1, 1, v, 1
    pe.ffn_backward(dy, None, gu, None, w2, dgu, h, dw2=dw2, act=act)
    torch.cuda.synchronize()
    a, rel = _act(vv, act), _rel(vv, act)
    s, e_s = _slope(vv, act), _slope_err(vv, act)
    for t in range(T):
        _within(_np(h)[t], a, np.abs(a) * (rel + BF * (1 + rel)), "h")
        _within(_np(dgu)[t, I:], a, np.abs(a) * (rel + BF * (1 + rel)), "du")
        _within(_np(dgu)[t, :I], s, e_s + BF * (np.abs(s) + e_s), "dg")
