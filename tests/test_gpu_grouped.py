"""GPU parity of the 4-bit products and of those grouped by expert against the 64-bit oracle (MI355X only).

Every tolerance is an error bound worked out per element from the arithmetic: an fp32 sum of n products is off by at most
(n + 8) * 2^-24 * sum |a| |b| whatever its order, an output is rounded once (bf16 2^-8, fp32 2^-24 of the value), and exp
and erf in fp32 are good to 2^-16 of the value over the inputs' range.  A product with int4 weights adds up x q and
-8 x, two terms of each k, of which |x| (q + 8) s is the size, and multiplies each sum over 128 of them by its scale: n =
2 K + K / 128.  Products with MXFP4 weights take the weights as they are, exactly.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gradient_bounds
import host_paged_expert_amd as pe
from oracle import dense, formats, grouped
from test_gpu_dense import BF, DEV, FN, GUARD, _backward_bounds, _bf, _np, _padded, _strided, _within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def _weights(rng, wtype, shape, sd=0.1):
    """Device weights and scales, their values, and the size of each weight's terms (see above)."""
    K = shape[-1]
    if wtype == "bf16":
        w, wv = _bf(rng.standard_normal(shape) * sd)
        return w, None, wv, np.abs(wv)
    codes = rng.integers(0, 256, shape[:-1] + (K // 2,)).astype(np.uint8)
    flat = codes.reshape(-1, K // 2)
    if wtype == "int4":
        s = (rng.random(shape[:-1] + (K // 128,)) * 0.02 + 0.005).astype(np.float16)
        bits = s.view(np.uint16).reshape(-1, K // 128)
        v = formats.dequant_int4_g128(flat, bits)
        size = (formats.unpack_int4(flat) + 8) * np.repeat(formats.f16_to_f32(bits).astype(np.float64), 128, 1)
        return (torch.from_numpy(codes).to(DEV), torch.from_numpy(s).to(DEV), v.reshape(shape).astype(np.float64),
                size.reshape(shape))
    s = rng.integers(119, 126, shape[:-1] + (K // 32,)).astype(np.uint8)
    v = formats.dequant_mxfp4_b32(flat, s.reshape(-1, K // 32)).reshape(shape).astype(np.float64)
    return torch.from_numpy(codes).to(DEV), torch.from_numpy(s).to(DEV), v, np.abs(v)


def _terms(wtype, K):
    return 2 * K + K // 128 if wtype == "int4" else K


def _k(wtype, K):
    step = {"bf16": 8, "int4": 128, "mxfp4": 32}[wtype]
    return max(step, K // step * step)


def _bound(x, size, n):
    """Error of every sum of the product of x and weights whose terms are of this size."""
    return (np.abs(x) @ size.T) * (n + 8) * U


def _check_linear(y, x, w, size, n, bias=None, act="none", residual=None, out_eps=BF, what="y"):
    e = _bound(x, size, n)
    pre = x @ w.T
    if bias is not None:
        pre = pre + bias
    e = e + U * (np.abs(pre) + e)
    ref = dense.act(pre, act)
    if act != "none":
        e = 1.13 * e + FN * (np.abs(ref) + 1.13 * e)
    if residual is not None:
        ref = ref + residual
        e = e + U * (np.abs(ref) + e)
    _within(y, ref, e + out_eps * (np.abs(ref) + e) + 1e-30, what)


def _check_glu(h, gu, x, w, size, n, act, what="h"):
    e = _bound(x, size, n)
    I = w.shape[0] // 2
    g, u, ref = dense.glu(x, w, act)
    a, e_g, e_u = np.abs(dense.act(g, act)), e[:, :I], e[:, I:]
    e_a = 1.13 * e_g + FN * (a + 1.13 * e_g)
    e_h = a * e_u + e_a * (np.abs(u) + e_u) + 2.0 ** -23 * np.abs(ref)
    _within(h, ref, e_h + BF * (np.abs(ref) + e_h) + 1e-30, what)
    if gu is not None:
        both = np.concatenate([g, u], 1)
        _within(gu, both, e + BF * (np.abs(both) + e) + 1e-30, "gu")


# ------------------------------------------------------------------ 4-bit products

# one row to many; columns that end inside a tile; k that ends inside a step, a scale's stretch (1024) or a stage
W4 = [(1, 16, 128), (1, 17, 256), (2, 1000, 1024), (3, 40, 96), (4, 2880, 2880), (8, 100, 640), (9, 24, 1152),
      (16, 513, 384), (17, 64, 160), (31, 130, 2176), (33, 257, 1056), (64, 96, 512), (65, 200, 1280), (127, 128, 1024),
      (129, 384, 2048), (257, 1000, 1120), (300, 129, 3200), (1, 8, 32), (40, 8, 32), (5, 6144, 512)]


@pytest.mark.parametrize("T,N,K", W4)
@pytest.mark.parametrize("wtype", ["int4", "mxfp4"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_linear_w4(T, N, K, wtype, dt):
    rng = np.random.default_rng(T * 31 + N + K)
    K = _k(wtype, K)
    x, xv = _bf(rng.standard_normal((T, K)))
    w, s, wv, size = _weights(rng, wtype, (N, K))
    act = ("none", "silu", "gelu")[(T + N) % 3]
    bias, bv = _bf(rng.standard_normal(N)) if T % 2 else (None, None)
    res, rv = _bf(rng.standard_normal((T, N))) if N % 2 == 0 else (None, None)
    out, ok = _padded(T, N, dt, pad=24 if N % 2 else 25, offset=T % 3)
    pe.linear_w4(_strided(x), w, s, out, bias=bias, act=act, residual=None if res is None else _strided(res))
    torch.cuda.synchronize()
    _check_linear(_np(out) if dt == torch.bfloat16 else out.cpu().numpy().astype(np.float64), xv, wv, size,
                  _terms(wtype, K), bv, act, rv, BF if dt == torch.bfloat16 else U)
    ok()


@pytest.mark.parametrize("T,I,H", [(1, 8, 128), (1, 768, 2048), (2, 40, 256), (4, 2880, 2880), (5, 64, 96), (16, 136, 640),
                                   (17, 24, 1152), (33, 200, 1056), (64, 64, 2176), (129, 72, 512), (256, 128, 1024),
                                   (300, 264, 1280)])
@pytest.mark.parametrize("wtype,act", [("int4", "silu"), ("mxfp4", "gelu")])
def test_glu_w4(T, I, H, wtype, act):
    rng = np.random.default_rng(T * 17 + I + H)
    H = _k(wtype, H)
    x, xv = _bf(rng.standard_normal((T, H)))
    w, s, wv, size = _weights(rng, wtype, (2 * I, H))
    out, ok = _padded(T, I, pad=24 if T % 2 else 23)
    pe.glu_w4(_strided(x), w, s, out, act=act)
    torch.cuda.synchronize()
    _check_glu(_np(out), None, xv, wv, size, _terms(wtype, H), act)
    ok()


@pytest.mark.parametrize("T", [1, 40, 130])
def test_every_code_and_scale(T):
    """x picks out single weights: all sixteen codes, every int4 scale's kind and every E8M0 byte up to where bf16 ends,
    exactly; from byte 253 on NaN."""
    K = 8192
    rng = np.random.default_rng(7)
    codes = np.tile(np.arange(256, dtype=np.uint8), (16, K // 512)).reshape(16, K // 2)
    bytes_ = np.tile(np.arange(256, dtype=np.uint8), (16, 1))
    at = rng.integers(0, 32, (T, 256)) + 32 * np.arange(256)
    values = formats.e2m1_to_f32(formats.unpack_int4(codes)).astype(np.float64)
    for t in range(0, T, 7):                                     # one weight at a time is the row of a one-hot x
        for blk in (0, 1, 2, 126, 127, 128, 250, 251, 252, 253, 254, 255, int(rng.integers(0, 255))):
            k = int(at[t, blk])
            x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
            x[t, k] = 1.0
            b = bytes_.copy()
            b[:, np.arange(256) != blk] = 127
            y = torch.empty((T, 16), dtype=torch.float32, device=DEV)
            pe.linear_w4(x, torch.from_numpy(codes).to(DEV), torch.from_numpy(b).to(DEV), y)
            torch.cuda.synchronize()
            got = y[t].cpu().numpy().astype(np.float64)
            want = values[:, k] * (2.0 ** (blk - 127) if blk < 255 else np.nan)
            if blk < 253:
                assert np.array_equal(got, want), (blk, got, want)
            else:              # the block holds codes of 6: 6 * 2^126 is infinite in bf16, and times a 0 of x NaN
                assert np.isnan(got).all()
    half = np.array([0, 1, 0x3FF, 0x400, 0x3C00, 0x7BFF, 0xBC00, 0x8001], np.uint16)     # zero, denormals, largest, negative
    s = np.tile(half, (16, K // 128 // 8))
    q = formats.unpack_int4(codes).astype(np.float64) - 8
    for g in range(8):
        k = 128 * (g + 8 * int(rng.integers(0, 8))) + int(rng.integers(0, 128))
        x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
        x[T - 1, k] = 1.0
        y = torch.empty((T, 16), dtype=torch.float32, device=DEV)
        pe.linear_w4(x, torch.from_numpy(codes).to(DEV), torch.from_numpy(s.view(np.float16)).to(DEV), y)
        torch.cuda.synchronize()
        assert np.array_equal(y[T - 1].cpu().numpy().astype(np.float64),
                              q[:, k] * formats.f16_to_f32(half[g:g + 1])[0].astype(np.float64)), g


# ------------------------------------------------------------------ order by expert

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (4, 8, 128), (7, 3, 5), (64, 8, 16), (65, 8, 1024), (513, 1, 3),
                                   (600, 8, 128), (1025, 4, 32), (3000, 7, 65)])
def test_group_rows(T, k, E):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    bad = rng.random((T, k)) < 0.1
    ids[bad] = rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1], bad.sum())
    o, r, p = grouped.group_rows(ids, E)
    offsets, rows, places = (torch.full(s, 77, dtype=torch.int32, device=DEV) for s in ((E + 1,), (T * k,), (T, k)))
    pe.group_rows(_i32(ids), offsets, rows, places)
    torch.cuda.synchronize()
    assert np.array_equal(offsets.cpu().numpy(), o) and np.array_equal(places.cpu().numpy(), p)
    rows = rows.cpu().numpy()
    assert np.array_equal(rows[:len(r)], r) and (rows[len(r):] == 77).all()


def test_group_rows_of_no_tokens_and_of_bad_ids():
    offsets = torch.full((9,), 77, dtype=torch.int32, device=DEV)
    e = torch.empty
    pe.group_rows(e((0, 4), dtype=torch.int32, device=DEV), offsets, e(0, dtype=torch.int32, device=DEV),
                  e((0, 4), dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert not offsets.any()
    ids, rows, places = _i32(np.full((3, 4), -1)), _i32(np.full(12, 77)), _i32(np.zeros((3, 4)))
    offsets.fill_(5)
    pe.group_rows(ids, offsets, rows, places)
    torch.cuda.synchronize()
    assert not offsets.any() and bool((places == -1).all()) and bool((rows == 77).all())


# ------------------------------------------------------------------ grouped products

# rows of each expert (none, one, a tile's edge, many, all in one), and rows behind the last
COUNTS = [([1], 0), ([0, 0, 3, 0], 2), ([2, 1, 0, 1, 4, 0], 0), ([16, 17, 0, 15], 5), ([0, 40], 0), ([33, 0, 64, 31, 1], 3),
          ([130, 0, 1, 127, 129], 7), ([0, 300, 0], 20), ([1] * 70 + [0] * 5, 0), ([257, 5, 90], 1),
          ([0] * 100 + [2, 0, 9] + [0] * 60 + [1], 4)]


def _groups(counts, behind, X, rng):
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(offsets[-1]) + behind
    rows = rng.integers(0, X, R).astype(np.int32)
    rows[offsets[-1]:] = 2 ** 31 - 1 if R % 2 else -5            # never looked at
    return offsets, rows, R


def _parts(offsets):
    for e in range(len(offsets) - 1):
        if offsets[e + 1] > offsets[e]:
            yield e, slice(offsets[e], offsets[e + 1])


@pytest.mark.parametrize("i", range(len(COUNTS)))
@pytest.mark.parametrize("N,K", [(40, 256), (129, 1152), (300, 136)])
@pytest.mark.parametrize("wtype", ["bf16", "int4", "mxfp4"])
def test_grouped_linear(i, N, K, wtype):
    counts, behind = COUNTS[i]
    rng = np.random.default_rng(i * 100 + N + K)
    K, E, X = _k(wtype, K), len(counts), 37
    offsets, rows, R = _groups(counts, behind, X, rng)
    gather = (i + N) % 2 == 0
    x, xv = _bf(rng.standard_normal((X if gather else R, K)))
    w, s, wv, size = _weights(rng, wtype, (E, N, K))
    bias, bv = _bf(rng.standard_normal((E, N))) if i % 2 else (None, None)
    dt = torch.float32 if i % 3 == 0 else torch.bfloat16
    out, ok = _padded(R, N, dt)
    pe.grouped_linear(_strided(x), w, out, _i32(offsets), rows=_i32(rows) if gather else None, w_scales=s, bias=bias,
                      act="silu" if i % 4 == 1 else "none")
    torch.cuda.synchronize()
    got = out.float().cpu().numpy().astype(np.float64)
    for e, p in _parts(offsets):
        _check_linear(got[p], xv[rows[p]] if gather else xv[p], wv[e], size[e], _terms(wtype, K),
                      None if bv is None else bv[e], "silu" if i % 4 == 1 else "none", None,
                      U if dt is torch.float32 else BF, "expert %d" % e)
    assert (got[offsets[-1]:] == GUARD).all()
    ok()


@pytest.mark.parametrize("i", range(len(COUNTS)))
@pytest.mark.parametrize("I,H", [(24, 256), (136, 1160)])
@pytest.mark.parametrize("wtype,act", [("bf16", "silu"), ("int4", "gelu"), ("mxfp4", "silu")])
def test_grouped_glu(i, I, H, wtype, act):
    counts, behind = COUNTS[i]
    rng = np.random.default_rng(i * 10 + I + H)
    H, E, X = _k(wtype, H), len(counts), 29
    offsets, rows, R = _groups(counts, behind, X, rng)
    gather = i % 2 == 0
    x, xv = _bf(rng.standard_normal((X if gather else R, H)))
    w, s, wv, size = _weights(rng, wtype, (E, 2 * I, H))
    out, ok = _padded(R, I, pad=24 if i % 3 else 21)
    gu = torch.full((R, 2 * I), GUARD, dtype=torch.bfloat16, device=DEV) if i % 3 else None
    pe.grouped_glu(_strided(x), w, out, _i32(offsets), rows=_i32(rows) if gather else None, w_scales=s, act=act, gu=gu)
    torch.cuda.synchronize()
    got, kept = _np(out), None if gu is None else _np(gu)
    for e, p in _parts(offsets):
        _check_glu(got[p], None if kept is None else kept[p], xv[rows[p]] if gather else xv[p], wv[e], size[e],
                   _terms(wtype, H), act, "expert %d" % e)
    assert (got[offsets[-1]:] == GUARD).all() and (kept is None or (kept[offsets[-1]:] == GUARD).all())
    ok()


@pytest.mark.parametrize("wtype", ["bf16", "int4", "mxfp4"])
def test_unusual_offsets_stay_in_bounds(wtype):
    """Offsets that do not ascend, or pass the rows there are, and rows of x that do not exist: whatever comes out, what
    surrounds the outputs stays, and the call after it is right."""
    rng = np.random.default_rng(3)
    E, N, K, R = 5, 72, 256, 50
    w, s, wv, size = _weights(rng, wtype, (E, N, K))
    x, xv = _bf(rng.standard_normal((R, K)))
    out, ok = _padded(R, N)
    for o in ([0, 40, 10, 60, 2 ** 31 - 1, -5], [-7, 20, 20, 20, 20, 1000], [50, 40, 30, 20, 10, 0], [9, 9, 9, 9, 9, 9]):
        pe.grouped_linear(x, w, out, _i32(o), rows=_i32(rng.integers(-2 ** 31, 2 ** 31, R)), w_scales=s)
        torch.cuda.synchronize()
        ok()
    o = [0, 0, 20, 20, 49, 50]
    pe.grouped_linear(x, w, out, _i32(o), w_scales=s)
    torch.cuda.synchronize()
    for e, p in _parts(o):
        _check_linear(_np(out)[p], xv[p], wv[e], size[e], _terms(wtype, K))


# ------------------------------------------------------------------ sum back to tokens

@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (3, 8, 128), (5, 3, 520), (17, 4, 2880), (40, 9, 1024), (2, 5, 4104), (9, 1, 256)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_and_its_gradients(T, k, H, weighted):
    rng = np.random.default_rng(T + k + H)
    R = T * k + 3
    y, yv = _bf(rng.standard_normal((R, H)))
    places = rng.permutation(R)[:T * k].reshape(T, k).astype(np.int32)
    lost = rng.random((T, k)) < 0.2
    places[lost] = rng.choice([-1, R, -2 ** 31, 2 ** 31 - 1], lost.sum())
    wv = rng.standard_normal((T, k)).astype(np.float32)
    w = torch.from_numpy(wv).to(DEV) if weighted else None
    wv = wv.astype(np.float64) if weighted else np.ones((T, k))
    res, rv = _bf(rng.standard_normal((T, H))) if T % 2 else (None, None)
    out, ok = _padded(T, H)
    pe.combine(_strided(y), _i32(places), out, topk_w=w, residual=None if res is None else _strided(res))
    torch.cuda.synchronize()
    size = grouped.combine(np.abs(yv), places, np.abs(wv), None if rv is None else np.abs(rv))
    ref = grouped.combine(yv, places, wv, rv)
    _within(_np(out), ref, BF * np.abs(ref) + size * (k + 2) * U * (1 + BF) + 1e-30)
    ok()

    dout, dv = _bf(rng.standard_normal((T, H)))
    dy, dy_ok = _padded(R, H)
    dw = torch.full((T, k), GUARD, device=DEV)
    pe.combine_backward(_strided(dout), _i32(places), dy, topk_w=w, y=_strided(y), dtopk_w=dw)
    torch.cuda.synchronize()
    ry, rw = grouped.combine_backward(dv, places, wv, yv)
    _, size = grouped.combine_backward(np.abs(dv), places, np.abs(wv), np.abs(yv))
    got = _np(dy)
    named = ~np.isnan(ry)
    _within(got[named], ry[named], np.abs(ry[named]) * (BF + 2.0 ** -23), "dy")
    assert (got[~named] == GUARD).all()
    _within(dw.cpu().numpy().astype(np.float64), rw, size * (H + 8) * U + 1e-30, "dw")
    dy_ok()
    # each by itself is the same
    dy2, dw2 = torch.full((R, H), GUARD, dtype=torch.bfloat16, device=DEV), torch.full_like(dw, GUARD)
    pe.combine_backward(dout, _i32(places), dy2, topk_w=w)
    pe.combine_backward(dout, _i32(places), topk_w=w, y=y, dtopk_w=dw2)
    torch.cuda.synchronize()
    assert torch.equal(dy2, dy) and torch.equal(dw2, dw)


def test_combine_special_rows():
    """A NaN or an infinity reaches the tokens that have its row and no other; a weight of a place that is none does
    not count, nor does its value."""
    T, k, H = 4, 2, 64
    rng = np.random.default_rng(0)
    y = _bf(rng.standard_normal((8, H)))[0]
    y[3, 5], y[6] = float("nan"), float("inf")
    places = _i32([[0, 1], [2, 3], [4, -1], [6, 7]])
    w = torch.tensor([[0.5, 0.5], [1.0, 1.0], [1.0, float("nan")], [0.25, 0.5]], device=DEV)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    pe.combine(y, places, out, topk_w=w)
    torch.cuda.synchronize()
    o = out.float().cpu()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all() and torch.isinf(o[3]).all()
    assert torch.isnan(o[1]).nonzero().flatten().tolist() == [5]
    same = y[:4].clone()
    pe.combine(y, places, same, topk_w=w, residual=same)         # in place
    pe.combine(y, places, out, topk_w=w, residual=y[:4].clone())
    torch.cuda.synchronize()
    assert torch.equal(same[[0, 2]], out[[0, 2]])
    e = torch.empty
    zero = torch.ones((2, H), dtype=torch.bfloat16, device=DEV)
    pe.combine(e((0, H), dtype=torch.bfloat16, device=DEV), _i32([[0], [-1]]), zero)
    torch.cuda.synchronize()
    assert not zero.any()


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("i", range(len(COUNTS)))
@pytest.mark.parametrize("H,I", [(64, 24), (200, 136), (264, 72)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_grouped_ffn_backward(i, H, I, act):
    counts, behind = COUNTS[i]
    rng = np.random.default_rng(i + H + I)
    E, X = len(counts), 31
    offsets, rows, R = _groups(counts, behind, X, rng)
    gather = (i + I) % 2 == 0
    x, xv = _bf(rng.standard_normal((X if gather else R, H)))
    w13, w13v = _bf(rng.standard_normal((E, 2 * I, H)) * 0.1)
    w2, w2v = _bf(rng.standard_normal((E, H, I)) * 0.1)
    dy, dyv = _bf(rng.standard_normal((R, H)))
    gu, guv = _bf(rng.standard_normal((R, 2 * I)))
    g = lambda *s: torch.full(s, GUARD, dtype=torch.bfloat16, device=DEV)     # noqa: E731
    dgu, h, d13, d2 = g(R, 2 * I), g(R, I), g(E, 2 * I, H), g(E, H, I)
    dx, ok = _padded(R, H)
    o, r = _i32(offsets), _i32(rows) if gather else None
    pe.grouped_ffn_backward(_strided(dy), _strided(x), gu, w13, w2, o, dgu, rows=r, h=h, dx=dx, dw13=d13, dw2=d2, act=act)
    torch.cuda.synchronize()
    for e in range(E):
        p = slice(offsets[e], offsets[e + 1])
        if p.start == p.stop:
            assert not d13[e].any() and not d2[e].any()
            continue
        refs, tols = _backward_bounds(xv[rows[p]] if gather else xv[p], w13v[e], w2v[e], dyv[p], guv[p], act)
        for name, got, ref, tol in zip(("dx", "dw13", "dw2"), (dx[p], d13[e], d2[e]), refs, tols):
            _within(_np(got), ref, tol, "%s of expert %d" % (name, e))
    for t in (dx, dgu, h):
        assert bool((t[int(offsets[-1]):] == GUARD).all())
    ok()
    # each gradient by itself is the same
    one = [g(R, H), g(E, 2 * I, H), g(E, H, I)]
    pe.grouped_ffn_backward(dy, None, gu, w13, w2, o, dgu, dx=one[0], act=act)
    pe.grouped_ffn_backward(dy, x, gu, None, w2, o, dgu, rows=r, dw13=one[1], act=act)
    pe.grouped_ffn_backward(dy, None, gu, None, w2, o, dgu, h=h, dw2=one[2], act=act)
    torch.cuda.synchronize()
    assert torch.equal(one[0][:int(offsets[-1])], dx[:int(offsets[-1])])
    assert torch.equal(one[1], d13) and torch.equal(one[2], d2)


def test_long_lists_of_rows():
    """More rows than the list of rows in LDS holds at once (2048), through it and in order."""
    H, I, X = 64, 24, 500
    counts = [2050, 0, 4500]
    rng = np.random.default_rng(11)
    offsets, rows, R = _groups(counts, 0, X, rng)
    x, xv = _bf(rng.standard_normal((X, H)))
    dy = _bf(rng.standard_normal((R, H)))[0]
    gu = _bf(rng.standard_normal((R, 2 * I)))[0]
    w13, w2 = _bf(rng.standard_normal((3, 2 * I, H)) * 0.1)[0], _bf(rng.standard_normal((3, H, I)) * 0.1)[0]
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)           # noqa: E731
    dgu, d13 = e(R, 2 * I), e(3, 2 * I, H)
    pe.grouped_ffn_backward(dy, x, gu, w13, w2, _i32(offsets), dgu, rows=_i32(rows), dw13=d13)
    torch.cuda.synchronize()
    left = _np(dgu)                                              # the product's own input
    for k, p in _parts(offsets):
        n = p.stop - p.start
        ref = left[p].T @ xv[rows[p]]
        err = (n + 8) * U * (np.abs(left[p]).T @ np.abs(xv[rows[p]]))
        _within(_np(d13[k]), ref, err + BF * (np.abs(ref) + err) + 1e-30, "expert %d" % k)


def test_no_rows():
    E, H, I = 3, 64, 24
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=DEV)    # noqa: E731
    o = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    pe.linear_w4(e(0, 128), e(8, 64, dt=torch.uint8), e(8, 1, dt=torch.float16), e(0, 8))
    pe.glu_w4(e(0, 128), e(16, 64, dt=torch.uint8), e(16, 1, dt=torch.float16), e(0, 8))
    pe.grouped_linear(e(0, H), e(E, 8, H), e(0, 8), o)
    pe.grouped_glu(e(0, H), e(E, 2 * I, H), e(0, I), o)
    pe.combine(e(0, H), e(0, 2, dt=torch.int32), e(0, H))
    pe.combine_backward(e(0, H), e(0, 2, dt=torch.int32), e(0, H))
    d13, d2 = (torch.full(s, GUARD, dtype=torch.bfloat16, device=DEV) for s in ((E, 2 * I, H), (E, H, I)))
    pe.grouped_ffn_backward(e(0, H), e(0, H), e(0, 2 * I), e(E, 2 * I, H), e(E, H, I), o, e(0, 2 * I), h=e(0, I), dx=e(0, H),
                            dw13=d13, dw2=d2)
    torch.cuda.synchronize()
    assert not d13.any() and not d2.any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(act):
    """Every coordinate of the gradients against the difference of the 64-bit forward at two points beside it."""
    T, H, I, E = 5, 16, 8, 3
    counts = [5, 0, 5]
    points = [gradient_bounds.point(T, H, I, act, e, lambda a: torch.from_numpy(a).to(torch.bfloat16).double().numpy())
              for e in range(E)]
    x, dy = (_bf(np.concatenate([points[e][i] for e in (0, 2)]))[0] for i in (0, 3))
    w13, w2 = (_bf(np.stack([p[i] for p in points]))[0] for i in (1, 2))
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)           # noqa: E731
    R, o = sum(counts), _i32(np.concatenate([[0], np.cumsum(counts)]))
    h, gu, dgu, h2, dx, d13, d2 = e(R, I), e(R, 2 * I), e(R, 2 * I), e(R, I), e(R, H), e(E, 2 * I, H), e(E, H, I)
    pe.grouped_glu(x, w13, h, o, act=act, gu=gu)
    pe.grouped_ffn_backward(dy, x, gu, w13, w2, o, dgu, h=h2, dx=dx, dw13=d13, dw2=d2, act=act)
    torch.cuda.synchronize()
    for n, k in enumerate((0, 2)):
        diffs, bounds = gradient_bounds.differences(*points[k], act), gradient_bounds.bounds(*points[k], act)
        for got, ref, tol in zip((dx[5 * n:5 * n + 5], d13[k], d2[k]), diffs, bounds):
            _within(_np(got), ref, tol, "expert %d" % k)
    assert not d13[1].any() and not d2[1].any()


# ------------------------------------------------------------------ on both sides of every choice of kernel

def _some(rng, n, count):
    return np.unique(np.concatenate([[0, n - 1, n // 2], rng.integers(0, n, count)]))


WAYS_LINEAR = [(1, 2048, 1152), (8, 4096, 1152), (8, 4104, 1152), (16, 6144, 1152), (16, 2048, 1152), (17, 700, 1024),
               (144, 2048, 1152), (150, 2048, 1152), (200, 2048, 2176), (500, 2048, 256), (1000, 2048, 256),
               (2048, 4096, 256), (2300, 4100, 384), (255, 33000, 128), (2048, 2048, 256), (2300, 2100, 384)]
WAYS_GLU = [(4, 768, 1152), (9, 768, 1152), (16, 776, 1152), (8, 8192, 256), (8, 8208, 256), (144, 1024, 1152),
            (200, 1024, 2176), (500, 1024, 256), (1000, 1024, 256), (2048, 2048, 256), (2300, 2056, 384), (2048, 1024, 256),
            (2300, 1032, 384)]


@pytest.mark.parametrize("T,N,K", WAYS_LINEAR)
@pytest.mark.parametrize("wtype", ["int4", "mxfp4"])
def test_linear_w4_where_its_ways_change(T, N, K, wtype):
    rng = np.random.default_rng(T + N + K)
    x, xv = _bf(rng.standard_normal((T, K)))
    w, s, wv, size = _weights(rng, wtype, (N, K))
    res, rv = _bf(rng.standard_normal((T, N)))
    out, ok = _padded(T, N)
    pe.linear_w4(x, w, s, out, residual=res)
    torch.cuda.synchronize()
    r, c = _some(rng, T, 60), _some(rng, N, 60)
    _check_linear(_np(out)[np.ix_(r, c)], xv[r], wv[c], size[c], _terms(wtype, K), residual=rv[np.ix_(r, c)])
    ok()


@pytest.mark.parametrize("T,I,H", WAYS_GLU)
@pytest.mark.parametrize("wtype", ["int4", "mxfp4"])
def test_glu_w4_where_its_ways_change(T, I, H, wtype):
    rng = np.random.default_rng(T + I + H)
    x, xv = _bf(rng.standard_normal((T, H)))
    w, s, wv, size = _weights(rng, wtype, (2 * I, H))
    out, ok = _padded(T, I)
    pe.glu_w4(x, w, s, out)
    torch.cuda.synchronize()
    r, c = _some(rng, T, 60), _some(rng, I, 60)
    both = np.concatenate([c, I + c])
    _check_glu(_np(out)[np.ix_(r, c)], None, xv[r], wv[both], size[both], _terms(wtype, H), "silu")
    ok()


# (experts, rows, columns, k): on average under 4 rows, up to 16, up to 96, more, 256 and more
WAYS_GROUPED = [(3, 5, 64, 1152), (32, 97, 96, 1152), (40, 100, 2048, 1152), (30, 80, 8208, 256), (5, 12, 100, 256),
                (4, 15, 200, 256), (4, 16, 200, 256), (4, 67, 200, 256), (4, 68, 200, 1152), (3, 290, 300, 256),
                (3, 294, 300, 1152), (200, 2000, 136, 128), (2, 1100, 6704, 256), (130, 300, 72, 128), (1024, 900, 40, 128),
                (2, 1100, 3400, 256)]


def _uneven(rng, E, R):
    """Offsets of E experts that share R rows unevenly, some with none."""
    cuts = np.sort(np.floor(R * rng.random(E - 1) ** 1.5).astype(np.int32))
    return np.concatenate([[0], cuts, [R]]).astype(np.int32)


@pytest.mark.parametrize("E,R,N,K", WAYS_GROUPED)
@pytest.mark.parametrize("wtype", ["bf16", "int4", "mxfp4"])
@pytest.mark.parametrize("glu", [False, True])
def test_grouped_products_where_their_ways_change(E, R, N, K, wtype, glu):
    rng = np.random.default_rng(E + R + N + K)
    N = N // 2 // 8 * 8 if glu else N
    F, X = (2 if glu else 1), 50
    offsets = _uneven(rng, E, R)
    rows = rng.integers(0, X, R).astype(np.int32)
    x, xv = _bf(rng.standard_normal((X, K)))
    w, s, wv, size = _weights(rng, wtype, (E, F * N, K))
    out, ok = _padded(R, N)
    if glu:
        pe.grouped_glu(x, w, out, _i32(offsets), rows=_i32(rows), w_scales=s)
    else:
        pe.grouped_linear(x, w, out, _i32(offsets), rows=_i32(rows), w_scales=s)
    torch.cuda.synchronize()
    got = _np(out)
    c = _some(rng, N, 50)
    both = np.concatenate([c, N + c]) if glu else c
    for e in np.unique(np.searchsorted(offsets, _some(rng, R, 12), side="right") - 1):
        p = np.arange(offsets[e], offsets[e + 1])
        p = p[_some(rng, len(p), 40)]
        if glu:
            _check_glu(got[np.ix_(p, c)], None, xv[rows[p]], wv[e][both], size[e][both], _terms(wtype, K), "silu")
        else:
            _check_linear(got[np.ix_(p, c)], xv[rows[p]], wv[e][c], size[e][c], _terms(wtype, K))
    ok()


@pytest.mark.parametrize("E,R,H,I", [(4, 387, 256, 136), (4, 388, 264, 128), (3, 700, 136, 264)])
def test_grouped_ffn_backward_where_its_ways_change(E, R, H, I):
    rng = np.random.default_rng(R)
    offsets = _uneven(rng, E, R)
    rows = rng.integers(0, 60, R).astype(np.int32)
    x, xv = _bf(rng.standard_normal((60, H)))
    w13, w13v = _bf(rng.standard_normal((E, 2 * I, H)) * 0.1)
    w2, w2v = _bf(rng.standard_normal((E, H, I)) * 0.1)
    dy, dyv = _bf(rng.standard_normal((R, H)))
    gu, guv = _bf(rng.standard_normal((R, 2 * I)))
    e = lambda *s: torch.full(s, GUARD, dtype=torch.bfloat16, device=DEV)     # noqa: E731
    dgu, h, dx, d13, d2 = e(R, 2 * I), e(R, I), e(R, H), e(E, 2 * I, H), e(E, H, I)
    pe.grouped_ffn_backward(dy, x, gu, w13, w2, _i32(offsets), dgu, rows=_i32(rows), h=h, dx=dx, dw13=d13, dw2=d2)
    torch.cuda.synchronize()
    for k, p in _parts(offsets):
        refs, tols = _backward_bounds(xv[rows[p]], w13v[k], w2v[k], dyv[p], guv[p], "silu")
        for name, got, ref, tol in zip(("dx", "dw13", "dw2"), (dx[p], d13[k], d2[k]), refs, tols):
            _within(_np(got), ref, tol, "%s of expert %d" % (name, k))


@pytest.mark.parametrize("T,k,E", [(128, 8, 70), (129, 8, 70), (16384, 8, 128), (16400, 8, 1024), (70000, 2, 3), (32768, 8, 128), (32800, 8, 1024)])
def test_group_rows_of_many_entries(T, k, E):
    rng = np.random.default_rng(T + k)
    ids = np.minimum(rng.integers(-1, E, (T, k)), rng.integers(0, E + 1, (T, k))).astype(np.int32)
    flat = ids.ravel()
    good = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(good, flat, E), kind="stable")[:good.sum()]
    places = np.full(T * k, -1, np.int32)
    places[order] = np.arange(len(order))
    offsets, rows, at = (torch.full(s, 77, dtype=torch.int32, device=DEV) for s in ((E + 1,), (T * k,), (T, k)))
    pe.group_rows(_i32(ids), offsets, rows, at)
    torch.cuda.synchronize()
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat[good], minlength=E))]))
    assert np.array_equal(at.cpu().numpy().ravel(), places)
    rows = rows.cpu().numpy()
    assert np.array_equal(rows[:len(order)], order // k) and (rows[len(order):] == 77).all()


# ------------------------------------------------------------------ matrices past 2^31 elements

def test_weights_and_rows_past_32_bits():
    """The last of many experts, rows of x and of y behind 2^31 elements, in the streaming kernels and in tiles."""
    rng = np.random.default_rng(1)
    E, N, K = 530, 1024, 4096                                    # 2.2e9 weights
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
    last, lv = _bf(rng.standard_normal((N, K)) * 0.1)
    w[E - 1] = last
    for R in (3, 2400):                                          # under 4 rows an expert, and more
        x, xv = _bf(rng.standard_normal((8, K)))
        o = np.zeros(E + 1, np.int32)
        o[E] = R
        o[E - 1] = R - 2
        o[1:E - 1] = R - 2
        rows = rng.integers(0, 8, R).astype(np.int32)
        y = torch.full((R, N), GUARD, dtype=torch.bfloat16, device=DEV)
        pe.grouped_linear(x, w, y, _i32(o), rows=_i32(rows))
        torch.cuda.synchronize()
        _check_linear(_np(y[R - 2:]), xv[rows[R - 2:]], lv, np.abs(lv), K)
        assert not y[:R - 2].any()
    del w
    big = torch.zeros((600, 4000000), dtype=torch.bfloat16, device=DEV)       # rows 4e6 elements apart
    x, y = big[:, :256], big[:, 1000000:1000064]
    xs, xv = _bf(rng.standard_normal((600, 256)))
    x.copy_(xs)
    ws, wv = _bf(rng.standard_normal((2, 64, 256)))
    pe.grouped_linear(x, ws, y, _i32([0, 599, 600]))
    torch.cuda.synchronize()
    _check_linear(_np(y[590:599]), xv[590:599], wv[0], np.abs(wv[0]), 256)
    _check_linear(_np(y[599:]), xv[599:], wv[1], np.abs(wv[1]), 256)
    q, s, qv, size = _weights(rng, "int4", (64, 256))
    pe.linear_w4(x, q, s, y)
    torch.cuda.synchronize()
    _check_linear(_np(y[590:]), xv[590:], qv, size, _terms("int4", 256))
    out = big[:, 2000000:2000256]
    pe.combine(x, _i32(np.arange(600)[::-1].reshape(600, 1)), out)
    torch.cuda.synchronize()
    assert torch.equal(out, x.flip(0))


def test_weight_gradients_past_32_bits():
    E, H, I = 270, 4096, 1024                                    # dw13: 2.3e9 elements
    rng = np.random.default_rng(2)
    dy, dyv = _bf(rng.standard_normal((5, H)))
    x, xv = _bf(rng.standard_normal((5, H)))
    gu, guv = _bf(rng.standard_normal((5, 2 * I)))
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device=DEV)
    last, lv = _bf(rng.standard_normal((H, I)) * 0.1)
    w2[E - 1] = last
    o = np.zeros(E + 1, np.int32)
    o[E] = 5
    d13 = torch.full((E, 2 * I, H), GUARD, dtype=torch.bfloat16, device=DEV)
    d2 = torch.full((E, H, I), GUARD, dtype=torch.bfloat16, device=DEV)
    dgu, h = torch.empty((5, 2 * I), dtype=torch.bfloat16, device=DEV), torch.empty((5, I), dtype=torch.bfloat16, device=DEV)
    pe.grouped_ffn_backward(dy, x, gu, None, w2, _i32(o), dgu, h=h, dw13=d13, dw2=d2)
    torch.cuda.synchronize()
    dguv, hv = _np(dgu), _np(h)                                  # the products' own inputs
    for got, left, right in ((d13[E - 1], dguv, xv), (d2[E - 1], dyv, hv)):
        r, n = _some(rng, left.shape[1], 40), _some(rng, right.shape[1], 40)
        ref = left[:, r].T @ right[:, n]
        err = 13 * U * (np.abs(left[:, r]).T @ np.abs(right[:, n]))
        _within(_np(got)[np.ix_(r, n)], ref, err + BF * (np.abs(ref) + err) + 1e-30)
    assert not d13[:E - 1].any() and not d2[:E - 1].any()


# ------------------------------------------------------------------ together

def _layer(T, E, k, H, I, seed):
    rng = np.random.default_rng(seed)
    mk = lambda *s, sd=1.0: _bf(rng.standard_normal(s) * sd)                  # noqa: E731
    return dict(x=mk(T, H), router=mk(E, H, sd=0.2), w13=mk(E, 2 * I, H, sd=0.1), w2=mk(E, H, I, sd=0.1), dout=mk(T, H))


def _forward_and_back(d, T, E, k, H, I, o, stream):
    """A routed block with its gradients, as a training step calls them."""
    x, router, w13, w2, dout = (d[n][0] for n in ("x", "router", "w13", "w2", "dout"))
    pe.linear(x, router, o["logits"], stream=stream)
    pe.route(o["logits"], o["ids"], o["w"], stream=stream)
    pe.group_rows(o["ids"], o["offsets"], o["rows"], o["places"], stream=stream)
    pe.grouped_glu(x, w13, o["h"], o["offsets"], rows=o["rows"], gu=o["gu"], stream=stream)
    pe.grouped_linear(o["h"], w2, o["y"], o["offsets"], stream=stream)
    pe.combine(o["y"], o["places"], o["out"], topk_w=o["w"], residual=x, stream=stream)
    pe.combine_backward(dout, o["places"], o["dy"], topk_w=o["w"], y=o["y"], dtopk_w=o["dw"], stream=stream)
    pe.grouped_ffn_backward(o["dy"], x, o["gu"], w13, w2, o["offsets"], o["dgu"], rows=o["rows"], h=o["h2"], dx=o["dxs"],
                            dw13=o["d13"], dw2=o["d2"], stream=stream)
    pe.combine(o["dxs"], o["places"], o["dx"], residual=dout, stream=stream)


def _buffers(T, E, k, H, I):
    e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=DEV)    # noqa: E731
    i, f, R = torch.int32, torch.float32, T * k
    return dict(logits=e(T, E, dt=f), ids=e(T, k, dt=i), w=e(T, k, dt=f), offsets=e(E + 1, dt=i), rows=e(R, dt=i),
                places=e(T, k, dt=i), h=e(R, I), gu=e(R, 2 * I), y=e(R, H), out=e(T, H), dy=e(R, H), dw=e(T, k, dt=f),
                dgu=e(R, 2 * I), h2=e(R, I), dxs=e(R, H), d13=e(E, 2 * I, H), d2=e(E, H, I), dx=e(T, H))


@pytest.mark.parametrize("T,E,k,H,I", [(5, 16, 4, 256, 96), (150, 8, 2, 264, 136), (1, 4, 1, 64, 8)])
def test_a_routed_block_and_its_gradients(T, E, k, H, I):
    """Route, group, multiply and combine, and back: against the block in 64 bits at the routing that was taken.  Every
    bf16 intermediate (h, y, dy, dgu, the rows of dx) is off by 2^-8 of itself and passes that on through the sums, in
    norm: the bounds are of whole rows or matrices, each intermediate's rounding with weight one of the result's norm
    times the widest spread that a sum of random signs leaves, 4."""
    d = _layer(T, E, k, H, I, T + E)
    o = _buffers(T, E, k, H, I)
    _forward_and_back(d, T, E, k, H, I, o, None)
    torch.cuda.synchronize()
    x, w13, w2, dout = (d[n][1] for n in ("x", "w13", "w2", "dout"))
    ids, w = o["ids"].cpu().numpy(), o["w"].cpu().numpy().astype(np.float64)
    offsets, rows, places = grouped.group_rows(ids, E)
    assert np.array_equal(o["offsets"].cpu().numpy(), offsets) and np.array_equal(o["rows"].cpu().numpy(), rows)
    R = T * k
    gu = grouped.linear(x, w13, None, "none", offsets, rows, R)
    h = dense.act(gu[:, :I], "silu") * gu[:, I:]
    y = grouped.linear(h, w2, None, "none", offsets, None, R)
    out = grouped.combine(y, places, w, x)
    dy, dw = grouped.combine_backward(dout, places, w, y)
    dxs, d13, d2 = np.zeros((R, H)), np.zeros((E, 2 * I, H)), np.zeros((E, H, I))
    for e, p in _parts(offsets):
        dxs[p], d13[e], d2[e] = dense.ffn_backward(dy[p], x[rows[p]], gu[p, :I], gu[p, I:], w13[e], w2[e], "silu")
    dx = grouped.combine(dxs, places, None, dout)
    for name, ref, steps in (("out", out, 4), ("dw", dw, 4), ("d13", d13, 5), ("d2", d2, 4), ("dx", dx, 6)):
        got = o[name].float().cpu().numpy().astype(np.float64)
        assert np.linalg.norm(got - ref) <= 4 * BF * steps * np.linalg.norm(ref), name


def test_captured_and_replayed():
    """The whole step captured once and replayed on new inputs (and so other experts' rows) between eager work."""
    T, E, k, H, I = 21, 12, 3, 128, 64
    d = _layer(T, E, k, H, I, 1)
    cap, eager = _buffers(T, E, k, H, I), _buffers(T, E, k, H, I)
    rng = np.random.default_rng(5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            _forward_and_back(d, T, E, k, H, I, cap, side)
    torch.cuda.synchronize()
    for _ in range(4):
        for n in ("x", "dout"):
            d[n][0].copy_(_bf(rng.standard_normal(d[n][0].shape))[0])
        g.replay()
        torch.cuda.synchronize()
        _forward_and_back(d, T, E, k, H, I, eager, torch.cuda.current_stream())
        torch.cuda.synchronize()
        for n in cap:
            assert torch.equal(cap[n], eager[n]), n


def test_two_streams_at_once_repeat_bit_for_bit():
    T, E, k, H, I = 64, 8, 2, 256, 128
    ds = [_layer(T, E, k, H, I, s) for s in (1, 2)]
    want = [_buffers(T, E, k, H, I) for _ in ds]
    for d, o in zip(ds, want):
        _forward_and_back(d, T, E, k, H, I, o, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [[_buffers(T, E, k, H, I) for _ in range(4)] for _ in ds]
    torch.cuda.synchronize()                                     # the buffers have been cleared
    for r in range(4):
        for d, o, s in zip(ds, got, streams):
            _forward_and_back(d, T, E, k, H, I, o[r], s)
    torch.cuda.synchronize()
    for a, runs in zip(want, got):
        for b in runs:
            for n in a:
                assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("wtype", ["int4", "mxfp4"])
def test_grouped_4bit_is_each_experts_own_product(wtype):
    """One expert's rows by linear_w4 and glu_w4, and all experts' by the grouped calls."""
    rng = np.random.default_rng(9)
    E, N, K, counts = 4, 96, 384, [3, 0, 50, 140]
    offsets, _, R = _groups(counts, 0, 1, rng)
    x, xv = _bf(rng.standard_normal((R, K)))
    w, s, wv, size = _weights(rng, wtype, (E, N, K))
    y, h = (torch.empty((R, n), dtype=torch.bfloat16, device=DEV) for n in (N, N // 2))
    pe.grouped_linear(x, w, y, _i32(offsets), w_scales=s)
    pe.grouped_glu(x, w, h, _i32(offsets), w_scales=s)
    for e, p in _parts(offsets):
        one, two = (torch.empty((p.stop - p.start, n), dtype=torch.bfloat16, device=DEV) for n in (N, N // 2))
        pe.linear_w4(x[p], w[e], s[e], one)
        pe.glu_w4(x[p], w[e], s[e], two)
        torch.cuda.synchronize()
        for got in (y[p], one):
            _check_linear(_np(got), xv[p], wv[e], size[e], _terms(wtype, K))
        for got in (h[p], two):
            _check_glu(_np(got), None, xv[p], wv[e], size[e], _terms(wtype, K), "silu")
