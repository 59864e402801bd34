"""The dense operators around a paged MoE layer.  TEST INFRASTRUCTURE (oracle).

Plain numpy in 64 bits over inputs already widened from their storage types;
nothing is rounded to the outputs' types except where an e4m3 code is the
output.  Formulas are those include/pe.h states.
"""
import math

import numpy as np

from . import formats

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126

_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(v, name):
    with np.errstate(over="ignore"):
        if name == "silu":
            return v / (1.0 + np.exp(-v))
        if name == "gelu":
            return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
    assert name == "none"
    return v


def act_grad(v, name):
    if name == "silu":
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    return 0.5 * (1.0 + _erf(v / math.sqrt(2.0))) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)


def rmsnorm(x, residual, weight, eps):
    """(v = x + residual, v / sqrt(mean(v^2) + eps) * weight)."""
    v = x.astype(np.float64) + (0.0 if residual is None else residual.astype(np.float64))
    return v, v / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps) * weight.astype(np.float64)


def group_scales(y):
    """[T, C/128]: max(largest magnitude of the group / 448, 2^-126)."""
    T, C = y.shape
    return np.maximum(np.abs(y).reshape(T, C // 128, 128).max(2) / E4M3_MAX, MIN_SCALE)


def dequant_rows(codes, scales):
    """e4m3 codes [T, C] times their scale per row and 128 columns."""
    return formats.e4m3_to_f32(codes).astype(np.float64) * np.repeat(scales.astype(np.float64), 128, axis=1)


def dequant_blocks(codes, scales):
    """e4m3 codes [N, K] times their scale per 128 x 128 block (the last block row may be short)."""
    s = np.repeat(np.repeat(scales.astype(np.float64), 128, axis=0)[:codes.shape[0]], 128, axis=1)
    return formats.e4m3_to_f32(codes).astype(np.float64) * s


def route(logits, k, scoring, renormalize, scale):
    """Row by row: ids of the k largest logits (ties to the lowest id; -inf and NaN never), weights."""
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        lg = [float(v) for v in logits[t]]
        ok = [e for e in range(E) if lg[e] == lg[e] and lg[e] != -math.inf]
        order = sorted(ok, key=lambda e: (-lg[e], e))[:k]
        if scoring == "softmax" and ok:
            m = max(lg[e] for e in ok)
            num = {e: 1.0 if lg[e] == m else math.exp(lg[e] - m) for e in ok}
            den = sum(num.values())
            score = {e: num[e] / den for e in ok}
        else:
            score = {e: 1.0 / (1.0 + math.exp(min(-lg[e], 700.0))) for e in ok}
        total = sum(score[e] for e in order)
        for r, e in enumerate(order):
            ids[t, r] = e
            w[t, r] = scale * (score[e] / total if renormalize and total > 0 else score[e])
    return ids, w


def linear(x, w, bias, act_name, residual):
    y = x @ w.T
    if bias is not None:
        y = y + bias
    y = act(y, act_name)
    return y if residual is None else y + residual


def glu(x, w13, act_name):
    """(g, u, act(g) * u)."""
    inter = w13.shape[0] // 2
    g, u = x @ w13[:inter].T, x @ w13[inter:].T
    return g, u, act(g, act_name) * u


def ffn_backward(dy, x, g, u, w13, w2, act_name):
    """(dx, dw13, dw2) of y = (act(g) * u) w2^T with g, u = x w13^T."""
    dh = dy @ w2
    a = act(g, act_name)
    dgu = np.concatenate([dh * u * act_grad(g, act_name), dh * a], axis=1)
    return dgu @ w13, dgu.T @ x, dy.T @ (a * u)
