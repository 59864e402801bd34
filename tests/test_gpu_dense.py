"""GPU parity of the dense operators against the 64-bit oracle (MI355X only).

Every tolerance is an error bound worked out per element from the arithmetic:
an fp32 sum of K products is off by at most (K + 8) * 2^-24 * sum |a| |b|
whatever its order, an output is rounded once (bf16 2^-8, e4m3 2^-4, fp32
2^-24 of the value), exp and erf in fp32 are good to 2^-16 of the value over
the inputs' range, and what goes through a bf16 intermediate carries that
rounding through the product after it.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import synth
import harness
import host_paged_expert_amd as pe
from oracle import dense, formats, moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F8 = 2.0 ** -8, 2.0 ** -4
FN = 2.0 ** -16          # exp / erf / division in fp32
GUARD = 77.0             # what surrounds an output and has to stay


def _bf(a):
    """numpy fp64 -> (device bf16, its exact values)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.float().numpy().astype(np.float64)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _codes(t):
    return t.detach().view(torch.uint8).cpu().numpy()


def _padded(rows, cols, dtype=torch.bfloat16, pad=24, offset=0):
    """A [rows, cols] view with row stride cols + pad into a buffer full of GUARD; `check` says
    whether everything around it stayed."""
    buf = torch.full((rows + 2, cols + pad), GUARD, dtype=dtype, device=DEV)
    view = buf[1:rows + 1, offset:offset + cols]

    def check():
        b = buf.float().clone()
        b[1:rows + 1, offset:offset + cols] = GUARD
        assert bool((b == GUARD).all()), "written outside the output"
    return view, check


def _strided(t, pad=16):
    """The same matrix with a longer row stride, NaN in the gaps."""
    if t.dtype == torch.bfloat16:
        buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    else:
        buf = torch.full((t.shape[0], t.shape[1] + pad), 0x7F, dtype=torch.uint8, device=DEV).view(t.dtype)
    v = buf[:, :t.shape[1]]
    v.copy_(t)
    return v


def _fp8_rows(rng, T, C):
    codes = rng.integers(0, 127, (T, C)).astype(np.uint8) | (rng.integers(0, 2, (T, C)) << 7).astype(np.uint8)
    scales = (rng.random((T, C // 128)) * 0.01 + 0.001).astype(np.float32)
    return codes, scales


def _fp8_blocks(rng, N, C):
    codes, _ = _fp8_rows(rng, N, C)
    return codes, (rng.random((-(-N // 128), C // 128)) * 0.001 + 0.0001).astype(np.float32)


def _dev8(codes):
    return torch.from_numpy(codes).to(DEV).view(torch.float8_e4m3fn)


def _aligned(x, w):
    """The FP8 term of every sum_k x[t,k] w[n,k]: 7 * 2^-13 times the largest |product| of each eight k, added up."""
    ax, aw = np.abs(x), np.abs(w)
    total = np.zeros((x.shape[0], w.shape[0]))
    for k in range(0, x.shape[1], 8):
        m = np.zeros_like(total)
        for j in range(k, k + 8):
            np.maximum(m, np.outer(ax[:, j], aw[:, j]), out=m)
        total += m
    return 7 * 2.0 ** -13 * total


def _within(got, ref, tol, what=""):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d outside, first at %s: got %r, want %r +- %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], ref[bad][0], np.broadcast_to(tol, got.shape)[bad][0])


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("T,H,quant", [(1, 8, False), (1, 128, True), (3, 136, False), (5, 2880, False),
                                       (7, 2048, True), (130, 640, True), (33, 4096, False), (2, 16384, False),
                                       (2, 16384, True), (1000, 1032, False), (1, 2048, True)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(T, H, quant, residual):
    rng = np.random.default_rng(T * 7 + H)
    x, xv = _bf(rng.standard_normal((T, H)) * 3)
    r, rv = _bf(rng.standard_normal((T, H)) * 2) if residual else (None, None)
    w, wv = _bf(1 + 0.1 * rng.standard_normal(H))
    x = _strided(x)
    v, y = dense.rmsnorm(xv, rv, wv, 1e-5)
    s, s_ok = _padded(T, H)
    # the mean of squares is a sum of positive numbers, off by (H/2) 2^-24 of itself at most; y has
    # half of that through the root, and five more fp32 operations
    rel = (H / 4 + 8) * 2.0 ** -24
    if quant:
        out = torch.full((T, H), 0x55, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        sc = torch.zeros((T, H // 128), device=DEV)
        pe.rmsnorm(x, w, 1e-5, out, scales=sc, residual=r, sum_out=s)
        torch.cuda.synchronize()
        want = dense.group_scales(y)
        _within(_np(sc), want, want * (rel + 2.0 ** -23), "scales")
        got = dense.dequant_rows(_codes(out), _np(sc))
        # half a step of the code (subnormal codes: 2^-10 of the scale), with y itself off by rel
        _within(got, y, np.abs(y) * (F8 * (1 + rel) + rel + 2.0 ** -22) + np.repeat(want, 128, 1) * 2.0 ** -9.9, "y")
    else:
        out, ok = _padded(T, H)
        pe.rmsnorm(x, w, 1e-5, out, residual=r, sum_out=s)
        torch.cuda.synchronize()
        _within(_np(out), y, np.abs(y) * (BF + 2 * rel), "y")
        ok()
    _within(_np(s), v, np.abs(v) * (BF + 2.0 ** -23), "sum")
    s_ok()


def test_rmsnorm_in_place_and_special_rows():
    """sum over the residual and y over x; a row of zeros, one with an infinity, one with a NaN, one of the
    smallest numbers and one of the largest leave the others as they are."""
    T, H = 8, 512
    rng = np.random.default_rng(1)
    a = rng.standard_normal((T, H))
    x, xv = _bf(a)
    r, rv = _bf(rng.standard_normal((T, H)))
    x[1], r[1] = 0, 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4], r[4] = 1e-38, 0
    w, wv = _bf(np.ones(H))
    xv, rv = _np(x), _np(r)
    v, y = dense.rmsnorm(xv, rv, wv, 1e-6)
    codes = torch.zeros((T, H), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((T, H // 128), device=DEV)
    pe.rmsnorm(x, w, 1e-6, codes, scales=sc, residual=r)
    pe.rmsnorm(x, w, 1e-6, x, residual=r, sum_out=r)
    torch.cuda.synchronize()
    fine = [0, 1, 4, 5, 6, 7]
    _within(_np(x)[fine], y[fine], np.abs(y[fine]) * (BF + 1e-4) + 1e-40, "y")
    _within(_np(r)[fine], v[fine], np.abs(v[fine]) * (BF + 1e-6) + 1e-40, "sum")
    assert np.isnan(_np(x)[3]).all()
    with np.errstate(invalid="ignore", over="ignore"):
        q = dense.dequant_rows(_codes(codes), _np(sc))
    assert np.isnan(q[3]).all() and (q[1] == 0).all() and (_np(sc)[1] == 2.0 ** -126).all()
    _within(q[fine], y[fine], np.abs(y[fine]) * (F8 + 1e-4) + np.repeat(_np(sc), 128, 1)[fine] * 2.0 ** -9.9, "codes")


@pytest.mark.parametrize("H", [256, 2048, 8192])
def test_rmsnorm_of_large_values(H):
    """Squares beyond fp32's range: the norm is still the formula's; ordinary rows beside them are not touched."""
    rng = np.random.default_rng(H)
    a = rng.standard_normal((5, H))
    a[1] *= 1e30
    a[3, 7] = 3e38
    x, xv = _bf(a)
    w, wv = _bf(1 + 0.1 * rng.standard_normal(H))
    _, y = dense.rmsnorm(xv, None, wv, 1e-6)
    out, ok = _padded(5, H)
    pe.rmsnorm(x, w, 1e-6, out)
    torch.cuda.synchronize()
    # two more fp32 operations than ordinary rows; what the scaled squares lose is below 2^-126 of a sum of 2^70 or more,
    # and an element of 1 beside 3e38 is a subnormal number times 2^70: an absolute error of 2^-80 at most
    _within(_np(out), y, np.abs(y) * (BF + (H / 2 + 20) * 2.0 ** -24) + 2.0 ** -80, "y")
    ok()


@pytest.mark.parametrize("H", [256, 2048])
@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_rmsnorm_of_small_values(H, eps):
    """Squares below fp32's range count where eps does not cover them; ordinary rows beside them, and a row of zeros
    under a positive eps, are as they were."""
    rng = np.random.default_rng(H + 1)
    a = rng.standard_normal((6, H))
    a[1] *= 1e-30
    a[2] *= 1e-36
    a[3] *= 1e-14
    if eps:
        a[4] = 0
    x, xv = _bf(a)
    w, wv = _bf(1 + 0.1 * rng.standard_normal(H))
    _, y = dense.rmsnorm(xv, None, wv, eps)
    out, ok = _padded(6, H)
    pe.rmsnorm(x, w, eps, out)
    torch.cuda.synchronize()
    # as for large values: the scalings by powers of two are exact, and the scaled squares of bf16 numbers are normal
    # (2^-133 at least becomes 2^-106)
    _within(_np(out), y, np.abs(y) * (BF + (H / 2 + 20) * 2.0 ** -24) + 1e-40, "y")
    ok()


# ------------------------------------------------------------------ routing

@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 7, 7), (4, 128, 8), (3, 64, 6), (9, 65, 3), (33, 32, 4),
                                   (2, 1024, 10), (1000, 128, 8), (7, 300, 300), (1, 256, 1)])
@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                            ("sigmoid", False)])
def test_route(T, E, k, scoring, renorm):
    rng = np.random.default_rng(T + E * 3 + k)
    lg = (rng.standard_normal((T, E)) * 3).astype(np.float32)
    lg[0] = np.round(lg[0])                         # ties: the lowest id first
    buf = torch.full((T, E + 3), float("nan"), device=DEV)
    buf[:, :E] = torch.from_numpy(lg).to(DEV)
    ids = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -7.0, device=DEV)
    pe.route(buf[:, :E], ids, w, scoring=scoring, renormalize=renorm, scale=2.5)
    torch.cuda.synchronize()
    want_ids, want = dense.route(lg, k, scoring, renorm, 2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # exp to 2^-21 of the value with arguments below 32, sums of at most 1024 positive terms
    _within(_np(w), want, want * (2.0 ** -19 + (E + k) * 2.0 ** -24), "weights")


def test_route_rows_without_choices():
    inf, nan = float("inf"), float("nan")
    rows = [[1, 3, 3, 2], [-inf, nan, 0, -inf], [-inf] * 4, [nan] * 4, [inf, 0, inf, 1], [-3.4e38] * 4, [-200] * 4]
    lg = np.array(rows, np.float32)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids = torch.full((len(rows), 3), -7, dtype=torch.int32, device=DEV)
            w = torch.full((len(rows), 3), -7.0, device=DEV)
            pe.route(torch.from_numpy(lg).to(DEV), ids, w, scoring=scoring, renormalize=renorm)
            torch.cuda.synchronize()
            want_ids, want = dense.route(lg, 3, scoring, renorm, 1.0)
            assert np.array_equal(ids.cpu().numpy(), want_ids)
            got = _np(w)
            if scoring == "sigmoid":
                # far below zero the sigmoid is under fp32's range (0) where 64 bits still have it:
                # those rows' weights are 0, renormalised or not
                want[5:] = 0.0
            _within(got, want, np.abs(want) * 2.0 ** -19, "weights")


# ------------------------------------------------------------------ products

SHAPES = [(1, 1, 8), (1, 128, 2048), (2, 7, 16), (3, 17, 8), (4, 2048, 768), (8, 33, 1000), (15, 64, 64), (16, 16, 72),
          (17, 33, 200), (31, 130, 136), (33, 260, 128), (63, 64, 192), (64, 100, 256), (65, 130, 200), (100, 515, 96),
          (127, 128, 64), (129, 257, 136), (257, 300, 1000), (200, 1200, 320), (513, 384, 512), (300, 2880, 2880)]


def _linear_case(T, N, K, fp8, rng):
    if fp8:
        K = max(128, K // 128 * 128)
        (xc, xs), (wc, ws) = _fp8_rows(rng, T, K), _fp8_blocks(rng, N, K)
        args = dict(x=_dev8(xc), w=_dev8(wc), x_scales=torch.from_numpy(xs).to(DEV),
                    w_scales=torch.from_numpy(ws).to(DEV))
        return args, dense.dequant_rows(xc, xs), dense.dequant_blocks(wc, ws), K
    x, xv = _bf(rng.standard_normal((T, K)))
    w, wv = _bf(rng.standard_normal((N, K)) * 0.1)
    return dict(x=x, w=w), xv, wv, K


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("fp8", [False, True])
def test_linear(T, N, K, fp8):
    rng = np.random.default_rng(T * 11 + N * 5 + K)
    args, xv, wv, K = _linear_case(T, N, K, fp8, rng)
    bias, bv = _bf(rng.standard_normal(N))
    res, rv = _bf(rng.standard_normal((T, N)))
    mag = np.abs(xv) @ np.abs(wv).T
    align = _aligned(xv, wv) if fp8 else 0.0
    args["x"] = _strided(args["x"])
    for act, with_bias, with_res, dt in [("none", False, False, torch.bfloat16), ("silu", True, True, torch.bfloat16),
                                         ("gelu", True, False, torch.float32), ("none", True, True, torch.float32),
                                         ("none", False, True, torch.bfloat16)]:
        out, ok = _padded(T, N, dt, pad=24 if act == "none" else 3)
        if act == "silu":                           # residual rows at an odd offset and stride
            rbuf = torch.zeros((T, N + 5), dtype=torch.bfloat16, device=DEV)
            rbuf[:, 1:N + 1] = res
            rt = rbuf[:, 1:N + 1]
        else:
            rt = res
        pe.linear(out=out, bias=bias if with_bias else None, act=act, residual=rt if with_res else None, **args)
        torch.cuda.synchronize()
        pre = dense.linear(xv, wv, bv if with_bias else None, "none", None)
        y = dense.act(pre, act) + (rv if with_res else 0.0)
        # both activations change by at most 1.13 of their argument's change
        err = 1.13 * ((K + 8) * 2.0 ** -24 * (mag + np.abs(pre)) + align) + FN * np.abs(dense.act(pre, act)) * (act != "none")
        tol = err + (BF if dt == torch.bfloat16 else 2.0 ** -23) * (np.abs(y) + err) + 2.0 ** -24 * np.abs(pre)
        _within(_np(out), y, tol, "%s %s" % (act, dt))
        ok()


@pytest.mark.parametrize("T,N,K", [(4096, 4096, 64), (4096, 4096, 136), (4095, 4099, 200), (2050, 12290, 72),
                                   (8192, 2048, 512), (1000, 9000, 64), (2048, 6144, 128)])
def test_linear_of_many_rows(T, N, K):
    """Enough output for the larger tiles: a sample of rows and columns, the edges among them, against the oracle."""
    rng = np.random.default_rng(T + N)
    x, xv = _bf(rng.standard_normal((T, K)))
    w, wv = _bf(rng.standard_normal((N, K)) * 0.1)
    bias, bv = _bf(rng.standard_normal(N))
    out, ok = _padded(T, N)
    pe.linear(x, w, out, bias=bias)
    torch.cuda.synchronize()
    ok()
    rows = np.unique(np.concatenate([[0, T - 1, 255 % T, 256 % T], rng.integers(0, T, 60)]))
    y = xv[rows] @ wv.T + bv
    err = (K + 8) * 2.0 ** -24 * (np.abs(xv[rows]) @ np.abs(wv).T + np.abs(y) + np.abs(bv))
    _within(_np(out)[rows], y, err + BF * (np.abs(y) + err))


@pytest.mark.parametrize("T,H,I", [(2048, 64, 6144), (2000, 136, 6152), (4096, 72, 2048), (4096, 64, 3000)])
def test_glu_of_many_rows(T, H, I):
    rng = np.random.default_rng(T + I)
    x, xv = _bf(rng.standard_normal((T, H)))
    w, wv = _bf(rng.standard_normal((2 * I, H)) * 0.1)
    out, ok = _padded(T, I)
    gu = torch.empty((T, 2 * I), dtype=torch.bfloat16, device=DEV)
    pe.glu(x, w, out, gu=gu)
    torch.cuda.synchronize()
    ok()
    rows = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 30)]))
    g, u, h = dense.glu(xv[rows], wv, "silu")
    mag = np.abs(xv[rows]) @ np.abs(wv).T * (H + 8) * 2.0 ** -24
    ag = np.abs(dense.act(g, "silu"))
    err = (1.13 * mag[:, :I] + FN * ag) * (np.abs(u) + mag[:, I:]) + ag * mag[:, I:] + 2.0 ** -23 * np.abs(h)
    _within(_np(out)[rows], h, err + BF * (np.abs(h) + err), "h")
    both = np.concatenate([g, u], 1)
    _within(_np(gu)[rows], both, mag + BF * (np.abs(both) + mag), "gu")


def test_ffn_backward_of_wide_weights():
    """Weight gradients large enough for the larger tiles over k-slow operands, with a ragged number of tokens."""
    T, H, I = 70, 2048, 6144
    dev, val = _backward_case(T, H, I, "silu", 17)
    x, w13, w2, dy, gu = dev
    xv, w13v, w2v, dyv, guv = val
    bufs = [torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((T, 2 * I), (T, I), (2 * I, H), (H, I))]
    pe.ffn_backward(dy, x, gu, w13, w2, bufs[0], bufs[1], dw13=bufs[2], dw2=bufs[3])
    torch.cuda.synchronize()
    dguv, hv = _np(bufs[0]), _np(bufs[1])              # the products' own inputs
    for got, left, right in ((bufs[2], dguv, xv), (bufs[3], dyv, hv)):
        ref = left.T @ right
        err = (T + 8) * 2.0 ** -24 * (np.abs(left).T @ np.abs(right))
        _within(_np(got), ref, err + BF * (np.abs(ref) + err) + 1e-30)
    g, u = guv[:, :I], guv[:, I:]
    h = dense.act(g, "silu") * u
    _within(hv, h, np.abs(h) * (BF + 2 * FN), "h")


def test_linear_into_its_residual():
    rng = np.random.default_rng(5)
    for T, N, K, fp8 in [(3, 100, 256, False), (200, 300, 256, False), (130, 256, 384, True)]:
        args, xv, wv, K = _linear_case(T, N, K, fp8, rng)
        res, rv = _bf(rng.standard_normal((T, N)))
        ref = torch.empty_like(res)
        pe.linear(out=ref, residual=res, **args)
        pe.linear(out=res, residual=res, **args)
        torch.cuda.synchronize()
        assert torch.equal(res, ref)


def _sample(rng, n, count):
    return np.unique(np.concatenate([[0, n - 1, n // 2], rng.integers(0, n, count)]))


# Sizes on both sides of every size at which the products change their way of working: few rows over narrow and wide
# weights, short and long sums, small, middling and large tiles.
CHANGES = [(1, 2040, 264), (4, 2056, 264), (2, 2600, 1032), (8, 2552, 136), (8, 2568, 136), (3, 4104, 1040),
           (7, 4104, 1000), (2, 8200, 72), (8, 8200, 1032), (9, 8200, 72), (16, 4096, 1152), (17, 2048, 1040),
           (32, 2056, 72), (300, 2048, 6144), (300, 2048, 4096), (500, 1024, 264), (512, 3000, 136),
           (1800, 2048, 136), (2048, 2048, 256), (2049, 2056, 200), (4099, 2300, 136), (2040, 2040, 200),
           (2048, 2880, 136), (1023, 2880, 200), (400, 2880, 2888), (1300, 2048, 1032)]


@pytest.mark.parametrize("T,N,K", CHANGES)
@pytest.mark.parametrize("fp8,dt", [(False, torch.bfloat16), (True, torch.bfloat16), (True, torch.float32)])
def test_linear_where_its_ways_change(T, N, K, fp8, dt):
    """A sample of rows and columns, the edges among them, against the oracle."""
    rng = np.random.default_rng(T + N + K)
    args, xv, wv, K = _linear_case(T, N, K, fp8, rng)
    out, ok = _padded(T, N, dt)
    pe.linear(out=out, **args)
    torch.cuda.synchronize()
    ok()
    rows, cols = _sample(rng, T, 12), _sample(rng, N, 60)
    xs, ws = xv[rows], wv[cols]
    y = xs @ ws.T
    err = (K + 8) * 2.0 ** -24 * (np.abs(xs) @ np.abs(ws).T + np.abs(y))
    if fp8 and dt == torch.bfloat16:
        err = err + _aligned(xs, ws)
    _within(_np(out)[rows][:, cols], y, err + (BF if dt == torch.bfloat16 else 2.0 ** -23) * (np.abs(y) + err), "y")


@pytest.mark.parametrize("T,H,I", [(1, 264, 1272), (4, 264, 1288), (2, 136, 2600), (8, 136, 2552), (8, 1040, 2568),
                                   (3, 2048, 6144), (9, 984, 608), (16, 1288, 2048), (16, 1280, 4096), (32, 72, 8192),
                                   (40, 72, 4104), (300, 264, 1536), (1000, 136, 3000), (2000, 136, 2048),
                                   (1000, 136, 1496), (2000, 136, 1016), (2048, 200, 1440), (400, 2888, 1440)])
@pytest.mark.parametrize("wtype,quant", [("bf16", False), ("bf16", True), ("fp8", False), ("fp8", True)])
def test_glu_where_its_ways_change(T, H, I, wtype, quant):
    rng = np.random.default_rng(T + H + I)
    if wtype == "fp8" or quant:
        I = I // 128 * 128
    args, xv, wv, H = _linear_case(T, 2 * I, H, wtype == "fp8", rng)
    args["w13"] = args.pop("w")
    rows = _sample(rng, T, 8)
    cols = np.concatenate([np.arange(0, 40), np.arange(I - 40, I)]) if not quant else np.concatenate(
        [np.arange(0, 128), np.arange(I - 128, I)])        # whole groups where the scales are checked
    xs, ws = xv[rows], wv[np.concatenate([cols, I + cols])]
    n = len(cols)
    g, u, h = dense.glu(xs, ws, "silu")
    wide = quant or wtype == "bf16"
    mag = np.abs(xs) @ np.abs(ws).T * (H + 8) * 2.0 ** -24 + (0.0 if wide else _aligned(xs, ws))
    ag = np.abs(dense.act(g, "silu"))
    err = (1.13 * mag[:, :n] + FN * ag) * (np.abs(u) + mag[:, n:]) + ag * mag[:, n:] + 2.0 ** -23 * np.abs(h)
    if not quant:
        out, ok = _padded(T, I)
        pe.glu(out=out, **args)
        torch.cuda.synchronize()
        ok()
        _within(_np(out)[rows][:, cols], h, err + BF * (np.abs(h) + err), "h")
        return
    out = torch.zeros((T, I), dtype=torch.float8_e4m3fn, device=DEV)
    sc = torch.zeros((T, I // 128), device=DEV)
    pe.glu(out=out, out_scales=sc, **args)
    torch.cuda.synchronize()
    got_s = _np(sc)[rows][:, [0, -1]]
    want = dense.group_scales(h)
    _within(got_s, want, err.reshape(len(rows), 2, 128).max(2) / 448 + want * 2.0 ** -22, "scales")
    got = dense.dequant_rows(_codes(out)[rows][:, cols], got_s)
    _within(got, h, err + F8 * (np.abs(h) + err) * (1 + 2.0 ** -20) + np.repeat(got_s, 128, 1) * 2.0 ** -9.9, "h")


def test_operands_and_outputs_in_columns_of_one_buffer():
    """x, the residual and y are column ranges of one buffer whose rows interleave; the rest of it stays as it was."""
    rng = np.random.default_rng(12)
    T, N, K = 37, 88, 64
    buf, bufv = _bf(rng.standard_normal((T, 256)))
    w, wv = _bf(rng.standard_normal((N, K)) / 8)
    x, r, y = buf[:, :K], buf[:, K:K + N], buf[:, K + N:K + 2 * N]
    pe.linear(x, w, y, residual=r)
    torch.cuda.synchronize()
    got = _np(buf)
    ref = bufv[:, :K] @ wv.T + bufv[:, K:K + N]
    tol = np.abs(ref) * BF + (np.abs(bufv[:, :K]) @ np.abs(wv).T + np.abs(bufv[:, K:K + N])) * (K + 2) * 2.0 ** -24 * (1 + BF)
    _within(got[:, K + N:K + 2 * N], ref, tol, "y")
    keep = np.r_[0:K + N, K + 2 * N:256]
    assert (got[:, keep] == bufv[:, keep]).all()
    g = torch.zeros((T, 64), dtype=torch.bfloat16, device=DEV)
    pe.rmsnorm(buf[:, :K], w[0], 1e-6, buf[:, 192:256])
    pe.rmsnorm(x, w[0], 1e-6, g)
    torch.cuda.synchronize()
    assert (_np(buf)[:, 192:] == _np(g)).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [2, 40, 150])
def test_rows_are_independent(T, fp8):
    """A NaN or infinite token row stays in its row, and no other row's bits change with it."""
    rng = np.random.default_rng(T)
    args, xv, wv, K = _linear_case(T, 200, 256, fp8, rng)
    a, b = (torch.empty((T, 200), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pe.linear(out=a, **args)
    if fp8:
        args["x"].view(torch.uint8)[1] = 0x7F
    else:
        args["x"][1] = float("inf")
        args["x"][1, 3] = float("nan")
    pe.linear(out=b, **args)
    torch.cuda.synchronize()
    assert torch.isnan(b[1]).all()
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("T,H,I", [(1, 64, 8), (1, 2048, 768), (2, 128, 128), (5, 2880, 200), (16, 256, 384),
                                   (17, 136, 136), (33, 512, 128), (64, 128, 640), (65, 256, 256), (130, 200, 328),
                                   (257, 384, 512), (300, 1024, 1152)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("wtype,quant", [("bf16", False), ("bf16", True), ("fp8", False), ("fp8", True)])
def test_glu(T, H, I, act, wtype, quant):
    rng = np.random.default_rng(T * 3 + H + I)
    fp8 = wtype == "fp8"
    if fp8 or quant:
        I = max(128, I // 128 * 128)
    args, xv, wv, H = _linear_case(T, 2 * I, H, fp8, rng)
    args["x"] = _strided(args["x"])
    args["w13"] = args.pop("w")
    g, u, h = dense.glu(xv, wv, act)
    mag = np.abs(xv) @ np.abs(wv).T * (H + 8) * 2.0 ** -24 + (_aligned(xv, wv) if fp8 else 0.0)
    dg, du = mag[:, :I], mag[:, I:]
    ag = np.abs(dense.act(g, act))
    err = (1.13 * dg + FN * ag) * (np.abs(u) + du) + ag * du + 2.0 ** -23 * np.abs(h)
    gu = torch.full((T, 2 * I), GUARD, dtype=torch.bfloat16, device=DEV)
    if quant:
        out = torch.zeros((T, I), dtype=torch.float8_e4m3fn, device=DEV)
        sc = torch.zeros((T, I // 128), device=DEV)
        pe.glu(out=out, out_scales=sc, act=act, gu=gu, **args)
        torch.cuda.synchronize()
        want = dense.group_scales(h)
        emax = err.reshape(T, I // 128, 128).max(2)
        _within(_np(sc), want, emax / 448 + want * 2.0 ** -22, "scales")
        got = dense.dequant_rows(_codes(out), _np(sc))
        _within(got, h, err + F8 * (np.abs(h) + err) * (1 + 2.0 ** -20) + np.repeat(_np(sc), 128, 1) * 2.0 ** -9.9, "h")
    else:
        out, ok = _padded(T, I, pad=24 if T % 2 else 3)
        pe.glu(out=out, act=act, gu=gu, **args)
        torch.cuda.synchronize()
        _within(_np(out), h, err + BF * (np.abs(h) + err), "h")
        ok()
    both = np.concatenate([g, u], 1)
    _within(_np(gu), both, mag + BF * (np.abs(both) + mag), "gu")
    out2, ok2 = _padded(T, I)
    if not quant:                                    # keeping gu does not change h
        pe.glu(out=out2, act=act, **args)
        torch.cuda.synchronize()
        assert torch.equal(out2, out)


def _backward_case(T, H, I, act, seed):
    rng = np.random.default_rng(seed)
    x, xv = _bf(rng.standard_normal((T, H)))
    w13, w13v = _bf(rng.standard_normal((2 * I, H)) * 0.1)
    w2, w2v = _bf(rng.standard_normal((H, I)) * 0.1)
    dy, dyv = _bf(rng.standard_normal((T, H)))
    gu, guv = _bf(xv @ w13v.T)
    return (x, w13, w2, dy, gu), (xv, w13v, w2v, dyv, guv)


def _backward_bounds(xv, w13v, w2v, dyv, guv, act):
    """The three gradients and the error bound of each element."""
    T, H = xv.shape
    I = w2v.shape[1]
    g, u = guv[:, :I], guv[:, I:]
    refs = dense.ffn_backward(dyv, xv, g, u, w13v, w2v, act)
    dh = dyv @ w2v
    e_dh = (np.abs(dyv) @ np.abs(w2v)) * (H + 8) * 2.0 ** -24
    a, slope = dense.act(g, act), dense.act_grad(g, act)
    # the slope is a sum of two terms of at most |1| and |1.13| magnitude, each good to FN
    e_slope = FN * 2.2
    dgu = np.concatenate([dh * u * slope, dh * a], 1)
    e_dgu = np.concatenate([np.abs(u) * (e_dh * (np.abs(slope) + e_slope) + np.abs(dh) * e_slope),
                            e_dh * np.abs(a) * (1 + FN) + np.abs(dh * a) * FN], 1)
    e_dgu = e_dgu + (BF + 2.0 ** -22) * (np.abs(dgu) + e_dgu)
    h = a * u
    e_h = np.abs(h) * (FN + BF * (1 + FN) + 2.0 ** -23)

    def product(p, e_p, q, n):
        """|p| q plus its errors: e_p q and the fp32 sum of n terms."""
        return e_p @ np.abs(q) + (np.abs(p) + e_p) @ np.abs(q) * (n + 8) * 2.0 ** -24
    e_dx = product(dgu, e_dgu, w13v, 2 * I)
    e_w13 = product(dgu.T, e_dgu.T, xv, T)
    e_w2 = (np.abs(dyv).T @ e_h) + (np.abs(dyv).T @ (np.abs(h) + e_h)) * (T + 8) * 2.0 ** -24
    return refs, [e + BF * (np.abs(r) + e) + 1e-30 for r, e in zip(refs, (e_dx, e_w13, e_w2))]


@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (1, 256, 128), (3, 64, 136), (16, 128, 64), (33, 200, 72), (64, 64, 256),
                                   (65, 136, 264), (127, 320, 128), (129, 256, 200), (257, 512, 384), (300, 264, 520)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_backward(T, H, I, act):
    dev, val = _backward_case(T, H, I, act, T + H)
    x, w13, w2, dy, gu = dev
    (rx, r13, r2), (tx, t13, t2) = _backward_bounds(*val, act)
    dgu = torch.full((T, 2 * I), GUARD, dtype=torch.bfloat16, device=DEV)
    h = torch.full((T, I), GUARD, dtype=torch.bfloat16, device=DEV)
    dx, ok = _padded(T, H)
    d13 = torch.full((2 * I, H), GUARD, dtype=torch.bfloat16, device=DEV)
    d2 = torch.full((H, I), GUARD, dtype=torch.bfloat16, device=DEV)
    pe.ffn_backward(_strided(dy), _strided(x), gu, w13, w2, dgu, h, dx=dx, dw13=d13, dw2=d2, act=act)
    torch.cuda.synchronize()
    _within(_np(dx), rx, tx, "dx")
    _within(_np(d13), r13, t13, "dw13")
    _within(_np(d2), r2, t2, "dw2")
    ok()
    # each gradient by itself is the same
    one = [torch.full_like(t, GUARD) for t in (dx, d13, d2)]
    pe.ffn_backward(dy, None, gu, w13, w2, dgu, dx=one[0], act=act)
    pe.ffn_backward(dy, x, gu, None, w2, dgu, dw13=one[1], act=act)
    pe.ffn_backward(dy, None, gu, None, w2, dgu, h, dw2=one[2], act=act)
    torch.cuda.synchronize()
    for a, b in zip(one, (dx, d13, d2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,H,I", [(5, 376, 1744), (132, 1184, 1456), (257, 2048, 768), (2169, 472, 504), (40, 720, 776),
                                   (691, 1000, 1000), (1100, 1024, 128)])
def test_ffn_backward_where_its_launches_change(T, H, I):
    """Few or many tiles in each of the three products, short and long sums, in one launch or apart."""
    dev, val = _backward_case(T, H, I, "silu", T + I)
    x, w13, w2, dy, gu = dev
    refs, tols = _backward_bounds(*val, "silu")
    dgu, h = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((T, 2 * I), (T, I)))
    out = [torch.full(s, GUARD, dtype=torch.bfloat16, device=DEV) for s in ((T, H), (2 * I, H), (H, I))]
    pe.ffn_backward(dy, x, gu, w13, w2, dgu, h, dx=out[0], dw13=out[1], dw2=out[2])
    torch.cuda.synchronize()
    for name, got, ref, tol in zip(("dx", "dw13", "dw2"), out, refs, tols):
        _within(_np(got), ref, tol, name)


def test_ffn_backward_of_no_tokens():
    H, I = 64, 32
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)          # noqa: E731
    d13, d2 = torch.full((2 * I, H), GUARD, dtype=torch.bfloat16, device=DEV), torch.full(
        (H, I), GUARD, dtype=torch.bfloat16, device=DEV)
    pe.ffn_backward(e(0, H), e(0, H), e(0, 2 * I), e(2 * I, H), e(H, I), e(0, 2 * I), e(0, I), dx=e(0, H), dw13=d13,
                    dw2=d2)
    torch.cuda.synchronize()
    assert bool((d13 == 0).all()) and bool((d2 == 0).all())


def test_no_tokens_and_byte_codes():
    """T = 0 through the tensor functions (weight gradients of larger tiles too), and e4m3 codes as bytes."""
    H, I = 2048, 6144
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=DEV)    # noqa: E731
    pe.rmsnorm(e(0, H), e(H), 1e-6, e(0, H))
    pe.route(e(0, 8, dt=torch.float32), e(0, 2, dt=torch.int32), e(0, 2, dt=torch.float32))
    pe.linear(e(0, H), e(16, H), e(0, 16))
    pe.glu(e(0, H), e(32, H), e(0, 16))
    d13 = torch.full((2 * I, H), GUARD, dtype=torch.bfloat16, device=DEV)
    d2 = torch.full((H, I), GUARD, dtype=torch.bfloat16, device=DEV)
    pe.ffn_backward(e(0, H), e(0, H), e(0, 2 * I), e(2 * I, H), e(H, I), e(0, 2 * I), e(0, I), dw13=d13, dw2=d2)
    torch.cuda.synchronize()
    assert bool((d13 == 0).all()) and bool((d2 == 0).all())
    rng = np.random.default_rng(0)
    args, *_ = _linear_case(20, 48, 256, True, rng)
    out = [e(20, 48) for _ in range(2)]
    pe.linear(out=out[0], **args)
    args["x"], args["w"] = args["x"].view(torch.uint8), args["w"].view(torch.uint8)
    pe.linear(out=out[1], **args)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1])


def test_a_refused_call_leaves_the_next_one_alone():
    x = torch.ones((2, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones((16, 64), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((2, 16), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(pe.PEError):
        pe.pe_linear(99, 0, x, 64, None, w, None, None, 0, None, 0, 2, 16, 64, y, 16, 0)     # no such device
    pe.linear(x, w, y)
    torch.cuda.synchronize()
    assert bool((y == 64).all())


def test_gradients_match_differences_of_the_forward():
    """dx, dw13 and dw2 of the kernels against central differences of the 64-bit forward at the kept gate and up
    values' own point: the loss moves along a direction by the gradient's product with it."""
    T, H, I, act = 6, 64, 48, "silu"
    dev, val = _backward_case(T, H, I, act, 3)
    x, w13, w2, dy, gu = dev
    xv, w13v, w2v, dyv, _ = val
    bufs = [torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((T, 2 * I), (T, I), (T, H), (2 * I, H), (H, I))]
    hh = torch.empty((T, I), dtype=torch.bfloat16, device=DEV)
    pe.glu(x, w13, hh, act=act, gu=gu)
    pe.ffn_backward(dy, x, gu, w13, w2, bufs[0], bufs[1], dx=bufs[2], dw13=bufs[3], dw2=bufs[4], act=act)
    torch.cuda.synchronize()
    grads = [_np(b) for b in bufs[2:]]

    def loss(p):
        return float((dense.glu(p[0], p[1], act)[2] @ p[2].T * dyv).sum())
    rng = np.random.default_rng(9)
    point, eps = [xv, w13v, w2v], 1e-4
    for i in range(3):
        for _ in range(5):
            d = rng.standard_normal(point[i].shape)
            up = [p + (eps * d if j == i else 0) for j, p in enumerate(point)]
            dn = [p - (eps * d if j == i else 0) for j, p in enumerate(point)]
            slope = (loss(up) - loss(dn)) / (2 * eps)
            # every element of a gradient is within a few bf16 roundings of intermediates of its size; in
            # the sum with a random direction they add as their magnitudes at most
            assert abs(slope - (grads[i] * d).sum()) <= 6 * BF * (np.abs(grads[i]) * np.abs(d)).sum()


# ------------------------------------------------------------------ streams, graphs, the block

def test_captured_and_replayed():
    """Every operator captured once in a graph, replayed with new inputs between eager work: each replay gives what
    the eager calls give."""
    T, H, I, E, k = 5, 256, 384, 16, 4
    rng = np.random.default_rng(2)
    mk = lambda *s, sd=1.0: _bf(rng.standard_normal(s) * sd)[0]               # noqa: E731
    x, res, nw = mk(T, H), mk(T, H), mk(H)
    wr, w13, w2, dy = mk(E, H, sd=0.1), mk(2 * I, H, sd=0.1), mk(H, I, sd=0.1), mk(T, H)
    e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=DEV)    # noqa: E731

    def outs():
        return dict(n=e(T, H), s=e(T, H), lg=e(T, E, dt=torch.float32), ids=e(T, k, dt=torch.int32),
                    w=e(T, k, dt=torch.float32), h=e(T, I), gu=e(T, 2 * I), y=e(T, H), dgu=e(T, 2 * I), h2=e(T, I),
                    dx=e(T, H), d13=e(2 * I, H), d2=e(H, I))

    def calls(o, st):
        pe.rmsnorm(x, nw, 1e-6, o["n"], residual=res, sum_out=o["s"], stream=st)
        pe.linear(o["n"], wr, o["lg"], stream=st)
        pe.route(o["lg"], o["ids"], o["w"], stream=st)
        pe.glu(o["n"], w13, o["h"], gu=o["gu"], stream=st)
        pe.linear(o["h"], w2, o["y"], residual=o["s"], stream=st)
        pe.ffn_backward(dy, o["n"], o["gu"], w13, w2, o["dgu"], o["h2"], dx=o["dx"], dw13=o["d13"], dw2=o["d2"],
                        stream=st)

    cap, eager = outs(), outs()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            calls(cap, side)
    torch.cuda.synchronize()
    for _ in range(4):
        for t in (x, res, dy):
            t.copy_(mk(*t.shape))
        g.replay()
        torch.cuda.synchronize()
        calls(eager, torch.cuda.current_stream())
        torch.cuda.synchronize()
        for n in cap:
            assert torch.equal(cap[n], eager[n]), n


def test_two_streams_at_once():
    """The same calls on two streams, with buffers of their own, do not disturb each other."""
    rng = np.random.default_rng(4)
    T, N, K = 40, 512, 1024
    w = _bf(rng.standard_normal((N, K)) * 0.1)[0]
    xs = [_bf(rng.standard_normal((T, K)))[0] for _ in range(2)]
    want = [torch.empty((T, N), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for i in range(2):
        pe.linear(xs[i], w, want[i])
    torch.cuda.synchronize()
    got = [[torch.zeros((T, N), dtype=torch.bfloat16, device=DEV) for _ in range(8)] for _ in range(2)]
    st = [torch.cuda.Stream() for _ in range(2)]
    for r in range(8):
        for i in range(2):
            pe.linear(xs[i], w, got[i][r], stream=st[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])


def test_results_repeat_bit_for_bit():
    rng = np.random.default_rng(6)
    for T in (1, 30, 300):
        args, *_ = _linear_case(T, 700, 640, False, rng)
        outs = [torch.empty((T, 700), device=DEV) for _ in range(3)]
        for o in outs:
            pe.linear(out=o, **args)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_moe_block_around_the_paged_layer():
    """Norm with residual, router, paged experts, shared expert and residual sum, as a decoder runs them, for a decode
    step and a prefill chunk: against the same block in 64 bits with the library's own routing."""
    wl = synth.workload("decode_bf16_k40_b1", layers=1, experts=16, top_k=4, resident=8, hidden=256, inter=256,
                        wtype="bf16", batch=1, steps=1)
    m = harness.make_moe(wl, max_tokens=40)
    harness.load_store(m, wl)
    cache = {}

    def expert(e):
        if e not in cache:
            cache[e] = formats.dequant_expert(wl.wtype, *synth.expert_tensors(wl, 0, e))
        return cache[e]
    rng = np.random.default_rng(8)
    H, I, E, k = wl.hidden, 512, wl.experts, wl.top_k
    nw, nwv = _bf(1 + 0.1 * rng.standard_normal(H))
    wr, wrv = _bf(rng.standard_normal((E, H)) * 0.1)
    w13, w13v = _bf(rng.standard_normal((2 * I, H)) * 0.05)
    w2, w2v = _bf(rng.standard_normal((H, I)) * 0.05)
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=DEV)    # noqa: E731
    for T in (1, 2, 40):
        x, xv = _bf(rng.standard_normal((T, H)))
        r, rv = _bf(rng.standard_normal((T, H)))
        n, s, lg, ids, w = e(T, H), e(T, H), e(T, E, dt=torch.float32), e(T, k, dt=torch.int32), e(T, k,
                                                                                                 dt=torch.float32)
        h, y, routed = e(T, I), e(T, H), e(T, H)
        pe.rmsnorm(x, nw, 1e-6, n, residual=r, sum_out=s)
        pe.linear(n, wr, lg)
        pe.route(lg, ids, w)
        m.forward(0, n, ids, w, routed)
        pe.glu(n, w13, h)
        pe.linear(h, w2, y, residual=s)
        pe.rmsnorm(y, nw, 1e-6, n, residual=routed, sum_out=y)      # the next layer's norm adds the routed part
        torch.cuda.synchronize()
        v, nv = dense.rmsnorm(xv, rv, nwv, 1e-6)
        want_ids, _ = dense.route(_np(lg).astype(np.float32), k, "softmax", True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        routed_v = moe.moe_layer(nv, want_ids, _np(w), expert, dtype=np.float64)
        total = v + dense.glu(nv, w13v, "silu")[2] @ w2v.T + routed_v
        # bf16 roundings of the normed row (twice through a product), of h, and of the three terms and their sums
        assert np.abs(_np(y) - total).max() <= 8 * BF * np.abs(total).max()
    m.close()


def test_fp8_chain_through_the_shared_expert():
    """Norm -> e4m3, glu FP8 -> e4m3, linear FP8 + residual: each step against the oracle on the step's own inputs."""
    rng = np.random.default_rng(12)
    T, H, I = 70, 256, 384
    x, xv = _bf(rng.standard_normal((T, H)))
    nw, nwv = _bf(np.ones(H))
    (c13, s13), (c2, s2) = _fp8_blocks(rng, 2 * I, H), _fp8_blocks(rng, H, I)
    q, qs = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((T, H // 128), device=DEV)
    h, hs = torch.empty((T, I), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((T, I // 128), device=DEV)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    d = lambda a: torch.from_numpy(a).to(DEV)                                 # noqa: E731
    pe.rmsnorm(x, nw, 1e-6, q, scales=qs)
    pe.glu(q, _dev8(c13), h, x_scales=qs, w_scales=d(s13), out_scales=hs)
    pe.linear(h, _dev8(c2), y, x_scales=hs, w_scales=d(s2), residual=x)
    torch.cuda.synchronize()
    qv, hv = dense.dequant_rows(_codes(q), _np(qs)), dense.dequant_rows(_codes(h), _np(hs))
    w13v, w2v = dense.dequant_blocks(c13, s13), dense.dequant_blocks(c2, s2)
    g, u, href = dense.glu(qv, w13v, "silu")
    # half an e4m3 step of each value, subnormal codes by their scale, and the products' own errors
    e = (H + 8) * 2.0 ** -24 * (np.abs(qv) @ np.abs(w13v).T) + _aligned(qv, w13v)
    ag = np.abs(dense.act(g, "silu"))
    eh = (1.13 * e[:, :I] + FN * ag) * (np.abs(u) + e[:, I:]) + ag * e[:, I:]
    _within(hv, href, F8 * (np.abs(href) + eh) * 1.001 + eh + np.repeat(_np(hs), 128, 1) * 2.0 ** -9.9, "h")
    yref = hv @ w2v.T + xv
    tol = (I + 8) * 2.0 ** -24 * 2 * (np.abs(hv) @ np.abs(w2v).T + np.abs(xv)) + _aligned(hv, w2v)
    tol = tol + BF * (np.abs(yref) + tol)
    _within(_np(y), yref, tol, "y")


def test_tensor_functions_refuse_what_does_not_match():
    T, H = 4, 256
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((128, H), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((T, 128), dtype=torch.bfloat16, device=DEV)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(w=w[:, :128]), dict(w=w.t()), dict(out=y[:, :100]),
                dict(out=y.half()), dict(bias=y[0, :100]), dict(residual=y.float()), dict(act="relu"),
                dict(x_scales=y.float()), dict(x=x[:, :128]), dict(x=torch.zeros((H, T), dtype=torch.bfloat16,
                                                                                 device=DEV).t()),
                dict(residual=y[:1].expand(T, 128))):
        kw = dict(x=x, w=w, out=y)
        kw.update(bad)
        with pytest.raises((ValueError, TypeError)):
            pe.linear(**kw)
    with pytest.raises(pe.PEError):
        pe.linear(x, w, x[:, :128])                 # the output lies in the input
    with pytest.raises(ValueError):
        pe.route(torch.zeros((T, 8), device=DEV), torch.zeros((T, 2), device=DEV), torch.zeros((T, 2), device=DEV))
