"""Gradients of the gated feed-forward block by differences of its 64-bit forward, one coordinate at a time, and how
far the library's may be from them.  TEST INFRASTRUCTURE."""
import numpy as np

from oracle import dense

BF = 2.0 ** -8
FN = 2.0 ** -16          # exp, erf and division in fp32
STEP = 1e-5


def point(T, H, I, act, seed, bf16):
    """x, w13, w2, dy as the library gets them (`bf16` rounds)."""
    rng = np.random.default_rng(seed)
    return [bf16(rng.standard_normal(s) * m) for s, m in
            (((T, H), 1.0), ((2 * I, H), 0.3), ((H, I), 0.3), ((T, H), 1.0))]


def differences(x, w13, w2, dy, act):
    """dx, dw13, dw2 of sum(dy * y): off by STEP^2 / 6 of the third derivative and 2^-52 |loss| / STEP."""
    def loss(x, w13, w2):
        return float((dense.glu(x, w13, act)[2] @ w2.T * dy).sum())
    args, grads = [x, w13, w2], []
    for i in range(3):
        g = np.empty(args[i].shape)
        for at in np.ndindex(*g.shape):
            keep = args[i][at]
            args[i][at] = keep + STEP
            up = loss(*args)
            args[i][at] = keep - STEP
            g[at] = (up - loss(*args)) / (2 * STEP)
            args[i][at] = keep
        grads.append(g)
    return grads


def bounds(x, w13, w2, dy, act):
    """For dx, dw13 and dw2, the error of each element where the library keeps g and u, dg and du and h as bf16 and
    rounds the gradients to bf16: every rounding at its largest, carried through the products."""
    T, H = x.shape
    I = w2.shape[1]
    g, u, h = dense.glu(x, w13, act)
    e_gu = np.abs(x) @ np.abs(w13).T * (H + 8) * 2.0 ** -24
    e_gu = e_gu + BF * (np.abs(np.concatenate([g, u], 1)) + e_gu)
    e_g, e_u = e_gu[:, :I], e_gu[:, I:]
    dh = np.abs(dy @ w2) + np.abs(dy) @ np.abs(w2) * (H + 8) * 2.0 ** -24
    e_dh = np.abs(dy) @ np.abs(w2) * (H + 8) * 2.0 ** -24
    a, slope = np.abs(dense.act(g, act)), np.abs(dense.act_grad(g, act))
    # |act'| <= 1.13; |act''| <= 0.5 for SiLU, 2 / sqrt(2 pi) for GELU
    e_a, e_s = 1.13 * e_g + FN * (a + 1.13 * e_g), 0.8 * e_g + 2.2 * FN
    e_dg = e_dh * np.abs(u) * slope + dh * (np.abs(u) * e_s + e_u * (slope + e_s))
    e_du = e_dh * a + dh * e_a
    dgu = np.concatenate([dh * np.abs(u) * slope, dh * a], 1)
    e_dgu = np.concatenate([e_dg, e_du], 1)
    e_dgu = e_dgu + BF * (dgu + e_dgu)
    e_h = a * e_u + e_a * (np.abs(u) + e_u)
    e_h = e_h + BF * (np.abs(h) + e_h)

    def product(p, e, q, n):
        return e @ np.abs(q) + (p + e) @ np.abs(q) * (n + 8) * 2.0 ** -24
    refs = dense.ffn_backward(dy, x, g, u, w13, w2, act)
    errs = (product(dgu, e_dgu, w13, 2 * I), product(dgu.T, e_dgu.T, x, T), product(np.abs(dy).T, 0 * dy.T, np.abs(h) + e_h, T) +
            np.abs(dy).T @ e_h)
    # and the differences' own error: third derivatives of order 100, a loss of order 100
    return [e + BF * (np.abs(r) + e) + 1e-6 for r, e in zip(refs, errs)]
