"""Matrices of more than 2^31 elements: rows before, at and after that offset against the 64-bit oracle (MI355X
only; some 20 GB of its memory)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import dense
from test_gpu_dense import BF, DEV, FN, _bf, _np, _within

pytestmark = pytest.mark.gpu
WIDE = 4112
T = 2 ** 31 // WIDE + 300                             # rows of WIDE columns, 2^31 elements and a few more


def _sample():
    at = 2 ** 31 // WIDE
    return np.unique(np.r_[0:3, 1000, at - 2:at + 3, T - 130, T - 2:T])


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _rows(cols, seed):
    """[T, cols] of the same 1024 random rows over and over, and the function that gives rows' exact values."""
    base, v = _bf(np.random.default_rng(seed).standard_normal((1024, cols)))
    x = _empty(T, cols)
    n = T // 1024 * 1024
    x[:n].view(-1, 1024, cols)[:] = base
    x[n:] = base[:T - n]
    return x, lambda r: v[r % 1024]


def test_norm():
    x, xv = _rows(WIDE, 1)
    w, wv = _bf(np.random.default_rng(2).standard_normal(WIDE))
    out = _empty(T, WIDE)
    pe.rmsnorm(x, w, 1e-6, out, sum_out=x)
    torch.cuda.synchronize()
    r = _sample()
    v, y = dense.rmsnorm(xv(r), None, wv, 1e-6)
    _within(_np(out[r]), y, np.abs(y) * (BF + (WIDE / 2 + 16) * 2.0 ** -24), "y")
    assert (_np(x[r]) == v).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_from_and_to_long_matrices(dtype):
    K = 64
    x, xv = _rows(K, 3)
    w, wv = _bf(np.random.default_rng(4).standard_normal((WIDE, K)) * 0.1)
    y = _empty(T, WIDE, dtype=dtype)
    pe.linear(x, w, y)
    torch.cuda.synchronize()
    r = _sample()
    ref = xv(r) @ wv.T
    err = (K + 8) * 2.0 ** -24 * (np.abs(xv(r)) @ np.abs(wv).T)
    _within(_np(y[r]), ref, err + (BF if dtype == torch.bfloat16 else 2.0 ** -23) * (np.abs(ref) + err), "y")
    if dtype == torch.bfloat16:                       # and back: the long matrix as x
        w2, w2v = _bf(np.random.default_rng(5).standard_normal((24, WIDE)) * 0.1)
        z = _empty(T, 24)
        pe.linear(y, w2, z, residual=z.zero_())
        torch.cuda.synchronize()
        yv = _np(y[r])
        ref = yv @ w2v.T
        err = (WIDE + 8) * 2.0 ** -24 * (np.abs(yv) @ np.abs(w2v).T)
        _within(_np(z[r]), ref, err + BF * (np.abs(ref) + err), "z")


def test_glu_and_its_gradients():
    H, I = 64, WIDE // 2                              # gu and dgu have WIDE columns
    x, xv = _rows(H, 6)
    w13, w13v = _bf(np.random.default_rng(7).standard_normal((2 * I, H)) * 0.1)
    w2, w2v = _bf(np.random.default_rng(8).standard_normal((H, I)) * 0.1)
    h, gu, dgu = _empty(T, I), _empty(T, 2 * I), _empty(T, 2 * I)
    pe.glu(x, w13, h, gu=gu)
    torch.cuda.synchronize()
    r = _sample()
    g, u, ref = dense.glu(xv(r), w13v, "silu")
    e = (H + 8) * 2.0 ** -24 * (np.abs(xv(r)) @ np.abs(w13v).T)
    both, ag = np.concatenate([g, u], 1), np.abs(dense.act(g, "silu"))
    _within(_np(gu[r]), both, e + BF * (np.abs(both) + e), "gu")
    err = (1.13 * e[:, :I] + FN * ag) * (np.abs(u) + e[:, I:]) + ag * e[:, I:] + 2.0 ** -23 * np.abs(ref)
    _within(_np(h[r]), ref, err + BF * (np.abs(ref) + err), "h")
    dx, dw13, dw2 = _empty(T, H), _empty(2 * I, H), _empty(H, I)
    pe.ffn_backward(x, x, gu, w13, w2, dgu, h, dx=dx, dw13=dw13, dw2=dw2)      # dy = x
    torch.cuda.synchronize()
    guv, dh = _np(gu[r]), xv(r) @ w2v
    g, u = guv[:, :I], guv[:, I:]
    ref = np.concatenate([dh * u * dense.act_grad(g, "silu"), dh * dense.act(g, "silu")], 1)
    e_dh = (H + 8) * 2.0 ** -24 * (np.abs(xv(r)) @ np.abs(w2v))
    err = np.concatenate([np.abs(u), np.abs(dense.act(g, "silu"))], 1) * (1.13 * np.tile(e_dh, 2) + 2.2 * FN * np.abs(
        np.tile(dh, 2))) + 2.0 ** -22 * np.abs(ref)
    _within(_np(dgu[r]), ref, err + BF * (np.abs(ref) + err), "dgu")
    dguv = _np(dgu[r])
    ref = dguv @ w13v
    err = (2 * I + 8) * 2.0 ** -24 * (np.abs(dguv) @ np.abs(w13v))
    _within(_np(dx[r]), ref, err + BF * (np.abs(ref) + err), "dx")
    # the weight gradients sum over all T rows: every 1024 of them give the same, exactly once per round
    cols = [0, 1, I - 1, I, 2 * I - 1]
    n, rest = T // 1024, T % 1024
    d, xs = _np(dgu[:1024][:, cols]), xv(np.arange(1024))
    times = n + (np.arange(1024) < rest)
    ref = (d * times[:, None]).T @ xs
    err = (T + 8) * 2.0 ** -24 * ((np.abs(d) * times[:, None]).T @ np.abs(xs))
    _within(_np(dw13[cols]), ref, err + BF * (np.abs(ref) + err), "dw13")
    hv = _np(h[:1024])
    ref = (xs[:, :4] * times[:, None]).T @ hv
    err = (T + 8) * 2.0 ** -24 * ((np.abs(xs[:, :4]) * times[:, None]).T @ np.abs(hv))
    _within(_np(dw2[:4]), ref, err + BF * (np.abs(ref) + err), "dw2")


def test_route():
    t, E, k = 2 ** 24 - 1, 160, 4                     # the most rows of one call: past 2^31 logits
    lg = torch.empty((t, E), device=DEV)
    base = np.random.default_rng(9).standard_normal((1024, E)).astype(np.float32)
    dev = torch.from_numpy(base).to(DEV)
    n = t // 1024 * 1024
    lg[:n].view(-1, 1024, E)[:] = dev
    lg[n:] = dev[:t - n]
    ids, w = _empty(t, k, dtype=torch.int32), _empty(t, k, dtype=torch.float32)
    pe.route(lg, ids, w)
    torch.cuda.synchronize()
    at = 2 ** 31 // E
    r = np.r_[0:3, at - 2:at + 3, t - 3:t]
    want_ids, want = dense.route(base[r % 1024], k, "softmax", True, 1.0)
    assert np.array_equal(ids[r].cpu().numpy(), want_ids)
    _within(_np(w[r]), want, want * (2.0 ** -19 + (E + k) * 2.0 ** -24), "weights")
