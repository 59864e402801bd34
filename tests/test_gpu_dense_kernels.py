"""The products' larger and rarer kernels against the 64-bit oracle (MI355X only): sizes that lead to each kernel
that the smaller tests do not reach.  A row of every 32 is checked over all its columns, the edges among them, so that
every tile has checked elements; tests/test_dense_launches.py holds the list against the library's own choices."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import dense
from test_gpu_dense import BF, DEV, FN, _aligned, _bf, _linear_case, _np, _padded, _within

pytestmark = pytest.mark.gpu

LINEAR = [(1438, 4979, 216), (1603, 4765, 328)]
GLU = [(3879, 136, 2088, False), (754, 328, 1104, False), (1001, 384, 2048, True),
       (2177, 256, 1024, True)]       # T, hidden, inter, FP8
BACKWARD = [(1795, 168, 3224, "x12"), (1795, 168, 3224, "1"), (1795, 168, 3224, "2"), (42, 792, 6056, "x12"),
            (2455, 1592, 144, "x12"), (4099, 2936, 136, "x"), (3313, 2520, 136, "x"), (1552, 4776, 136, "x"),
            (1133, 1896, 1344, "x12"), (1125, 872, 2736, "x12"), (150, 1384, 4920, "x12"), (4095, 2040, 2056, "x12")]


def _rows(rng, n):
    """0, n - 1 and one of every 32."""
    r = np.arange(0, n, 32) + rng.integers(0, 32, -(-n // 32))
    return np.unique(np.concatenate([[0, n - 1], r[r < n]]))


@pytest.mark.parametrize("T,N,K", LINEAR)
@pytest.mark.parametrize("fp32", [False, True])
def test_linear_kernels(T, N, K, fp32):
    rng = np.random.default_rng(T)
    x, xv = _bf(rng.standard_normal((T, K)))
    w, wv = _bf(rng.standard_normal((N, K)) * 0.1)
    bias, bv = _bf(rng.standard_normal(N))
    res, rv = _bf(rng.standard_normal((T, N)))
    out, ok = _padded(T, N, torch.float32 if fp32 else torch.bfloat16)
    pe.linear(x, w, out, bias=bias, residual=res)
    torch.cuda.synchronize()
    ok()
    rows = _rows(rng, T)
    y = xv[rows] @ wv.T + bv + rv[rows]
    err = (K + 8) * 2.0 ** -24 * (np.abs(xv[rows]) @ np.abs(wv).T + np.abs(bv) + np.abs(rv[rows]))
    _within(_np(out)[rows], y, err + (2.0 ** -23 if fp32 else BF) * (np.abs(y) + err), "y")


@pytest.mark.parametrize("T,H,I,fp8", GLU)
def test_glu_kernels(T, H, I, fp8):
    rng = np.random.default_rng(T)
    args, xv, wv, H = _linear_case(T, 2 * I, H, fp8, rng)
    args["w13"] = args.pop("w")
    out, ok = _padded(T, I)
    gu = torch.zeros((T, 2 * I), dtype=torch.bfloat16, device=DEV)
    pe.glu(out=out, gu=gu, **args)
    torch.cuda.synchronize()
    ok()
    rows = _rows(rng, T)
    g, u, h = dense.glu(xv[rows], wv, "silu")
    mag = np.abs(xv[rows]) @ np.abs(wv).T * (H + 8) * 2.0 ** -24
    if fp8:
        mag = mag + _aligned(xv[rows], wv)
    ag = np.abs(dense.act(g, "silu"))
    err = (1.13 * mag[:, :I] + FN * ag) * (np.abs(u) + mag[:, I:]) + ag * mag[:, I:] + 2.0 ** -23 * np.abs(h)
    _within(_np(out)[rows], h, err + BF * (np.abs(h) + err), "h")
    both = np.concatenate([g, u], 1)
    _within(_np(gu)[rows], both, mag + BF * (np.abs(both) + mag), "gu")


@pytest.mark.parametrize("T,H,I,which", BACKWARD)
def test_backward_kernels(T, H, I, which):
    """dgu and h against the formula, each gradient against the product of the dgu and h that it read."""
    rng = np.random.default_rng(T + I)
    x, xv = _bf(rng.standard_normal((T, H)))
    w13, w13v = _bf(rng.standard_normal((2 * I, H)) * 0.1)
    w2, w2v = _bf(rng.standard_normal((H, I)) * 0.1)
    dy, dyv = _bf(rng.standard_normal((T, H)))
    gu, guv = _bf(rng.standard_normal((T, 2 * I)))
    e = lambda *s: torch.full(s, 77.0, dtype=torch.bfloat16, device=DEV)      # noqa: E731
    dgu, h = e(T, 2 * I), e(T, I)
    dx, ok = _padded(T, H)
    d13, d2 = e(2 * I, H), e(H, I)
    pe.ffn_backward(dy, x, gu, w13, w2, dgu, h, dx=dx if "x" in which else None, dw13=d13 if "1" in which else None,
                    dw2=d2 if "2" in which else None)
    torch.cuda.synchronize()
    ok()
    dguv, hv = _np(dgu), _np(h)
    r = _rows(rng, T)
    dh = dyv[r] @ w2v
    e_dh = np.abs(dyv[r]) @ np.abs(w2v) * (H + 8) * 2.0 ** -24
    g, u = guv[r][:, :I], guv[r][:, I:]
    a, slope = dense.act(g, "silu"), dense.act_grad(g, "silu")
    ref = np.concatenate([dh * u * slope, dh * a], 1)
    err = np.concatenate([np.abs(u) * (e_dh * (np.abs(slope) + 2.2 * FN) + np.abs(dh) * 2.2 * FN),
                          e_dh * np.abs(a) * (1 + FN) + np.abs(dh * a) * FN], 1) + 2.0 ** -22 * np.abs(ref)
    _within(dguv[r], ref, err + BF * (np.abs(ref) + err), "dgu")
    if "2" in which:
        _within(hv[r], a * u, np.abs(a * u) * (BF + 2 * FN), "h")

    def product(name, got, left, right):               # rows of `got` = left^T right, given in its rows
        y = left @ right
        err = (left.shape[1] + 8) * 2.0 ** -24 * (np.abs(left) @ np.abs(right))
        _within(got, y, err + BF * (np.abs(y) + err) + 1e-30, name)
    if "x" in which:
        product("dx", _np(dx)[r], dguv[r], w13v)
    if "1" in which:
        r = _rows(rng, 2 * I)
        product("dw13", _np(d13)[r], dguv[:, r].T, xv)
    if "2" in which:
        r = _rows(rng, H)
        product("dw2", _np(d2)[r], dyv[:, r].T, hv)
