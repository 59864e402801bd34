"""The 4-bit products at the ends of their inputs' ranges, of every code and scale, and of MXFP4 rows that end inside a
step, in the kernels of few rows and in every tile (MI355X only).

The shapes say which kernel a call takes; test_four_bit_launches.py holds them to it.  An int4 product adds up
x (q - 8) / 16, each term exact, 128 of them at a time, and those sums times 16 s (exact in fp32): an fp32 result is off by
at most (K + K / 128 + 8) * 2^-24 * sum |x (q - 8) s|, and a single weight's product (8 + 4 + 11 bits) not at all.  MXFP4
weights are bf16 numbers, so a single one is exact too, and sums are off by at most (K + 8) * 2^-24 * sum |x w|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import formats
from test_gpu_dense import BF, DEV, FN, GUARD, _bf, _np, _padded, _within
from test_gpu_grouped import U, _check_glu, _check_linear, _i32, _parts, _some, _uneven, _weights

pytestmark = pytest.mark.gpu

# (rows, columns, k) of linear_w4
INT4_LINEAR = [(3, 40, 256), (1, 2048, 1152), (16, 6144, 1152), (16, 2048, 1152), (150, 2048, 1152), (500, 2048, 256),
               (2048, 2048, 256), (2300, 4100, 256)]
# (rows, columns, k) of glu_w4
INT4_GLU = [(5, 24, 256), (9, 768, 1152), (8, 8208, 256), (150, 1088, 1152), (500, 1024, 256), (2048, 1024, 256),
            (2300, 2056, 256)]
# (experts, rows, columns, k) of the grouped products
INT4_GROUPED = [(4, 9, 40, 1152), (3, 14, 200, 256), (3, 294, 136, 1152), (2, 1100, 3400, 256), (2, 1100, 6704, 256)]
# The same of MXFP4, in tiles: k shorter than a step (128), that end in each of its quarters, and just past a stretch of
# scales (1024).
MX_LINEAR = [(150, 2048, 1056), (150, 2048, 96), (200, 2048, 2880), (500, 2048, 160), (500, 2048, 1120), (1000, 2048, 32),
             (2048, 2048, 288), (2048, 2048, 1056), (2300, 4100, 96), (2300, 4100, 1120)]
MX_GLU = [(200, 1024, 2880), (150, 1088, 32), (500, 1024, 96), (500, 1024, 1056), (2048, 1024, 160), (2048, 1024, 1120),
          (2300, 2056, 1056), (2300, 2056, 64)]
MX_GROUPED = [(100, 700, 300, 1120), (100, 700, 300, 96), (4, 16, 200, 1120), (4, 16, 200, 32), (3, 14, 72, 2880), (3, 294, 300, 2880), (3, 294, 300, 96),
              (5, 300, 136, 1056), (2, 1100, 3400, 160), (2, 1100, 3400, 1056), (2, 1100, 6704, 96), (2, 1100, 6704, 1120)]


def _int4(rng, shape, codes=None):
    """Codes (at random, or these) and scales of int4 weights on the device, and their values."""
    K = shape[-1]
    if codes is None:
        codes = rng.integers(0, 16, shape)
    packed = (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)
    s = (rng.random(shape[:-1] + (K // 128,)) * 0.02 + 0.005).astype(np.float16)
    v = formats.dequant_int4_g128(packed.reshape(-1, K // 2), s.view(np.uint16).reshape(-1, K // 128))
    return torch.from_numpy(packed).to(DEV), torch.from_numpy(s).to(DEV), v.reshape(shape).astype(np.float64)


def _rows_checked(rng, T, special):
    return np.unique(np.concatenate([special, _some(rng, T, 20)])).astype(int)


def _hold(y, x, w, n, what):
    """fp32 or bf16 results: finite ones by the bound, the others alike."""
    with np.errstate(invalid="ignore"):
        ref = np.stack([(r * w).sum(1) for r in x])
        size = np.stack([(np.abs(r) * np.abs(w)).sum(1) for r in x])
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(y), np.isnan(ref)), what
    assert np.array_equal(y[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)]), what
    eps = U if y.dtype == np.float32 else BF
    e = size[fin] * (n + 8) * U
    _within(y[fin].astype(np.float64), ref[fin], e + eps * (np.abs(ref[fin]) + e) + 1e-30, what)


def _infinities(rng, T, K):
    """Rows of ordinary numbers, some with an infinity, two, or a NaN; and which."""
    x = rng.standard_normal((T, K))
    rows = np.unique([0, T // 2, T - 1])
    x[0, K - 1] = np.inf
    x[T // 2, 5] = -np.inf
    x[T - 1, 0], x[T - 1, K // 2] = np.inf, -np.inf
    if T > 8:
        x[7, 100] = np.nan
        rows = np.unique(np.append(rows, 7))
    return x, rows


def _large(rng, T, K):
    """Rows of numbers up to 2^121: 128 of them times 8 / 16 are below fp32's largest."""
    return rng.choice([-1.0, 1.0], (T, K)) * (0.5 + 0.5 * rng.random((T, K))) * 2.0 ** 121, np.array([0])


@pytest.mark.parametrize("T,N,K", INT4_LINEAR)
@pytest.mark.parametrize("make", [_infinities, _large])
def test_int4_products_of_infinities_and_of_large_rows(T, N, K, make):
    """Each result is what its own products add up to: an infinity gives one of the weight's sign and a NaN with a weight
    of zero, and rows whose sum of 15 |x| passes fp32's range have finite results."""
    rng = np.random.default_rng(T + N + K)
    x, special = make(rng, T, K)
    x, xv = _bf(x)
    w, s, wv = _int4(rng, (N, K))
    y = torch.empty((T, N), device=DEV)
    pe.linear_w4(x, w, s, y)
    torch.cuda.synchronize()
    r, c = _rows_checked(rng, T, special), _some(rng, N, 60)
    _hold(y.cpu().numpy()[np.ix_(r, c)], xv[r], wv[c], K + K // 128, "linear_w4")


@pytest.mark.parametrize("E,R,N,K", INT4_GROUPED)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("make", [_infinities, _large])
def test_grouped_int4_products_of_infinities_and_of_large_rows(E, R, N, K, glu, make):
    rng = np.random.default_rng(E + R + N + K)
    N = N // 2 // 8 * 8 if glu else N
    offsets = _uneven(rng, E, R)
    x, special = make(rng, R, K)
    x, xv = _bf(x)
    w, s, wv = _int4(rng, (E, (2 if glu else 1) * N, K))
    if glu:
        h, y = (torch.empty((R, n * N), dtype=torch.bfloat16, device=DEV) for n in (1, 2))
        pe.grouped_glu(x, w, h, _i32(offsets), w_scales=s, gu=y)             # gu: the products themselves
    else:
        y = torch.empty((R, N), device=DEV)
        pe.grouped_linear(x, w, y, _i32(offsets), w_scales=s)
    torch.cuda.synchronize()
    got, r, c = y.float().cpu().numpy(), _rows_checked(rng, R, special), _some(rng, wv.shape[1], 60)
    got = got.astype(np.float64) if glu else got
    of = np.searchsorted(offsets, r, side="right") - 1
    for e in np.unique(of):
        p = r[of == e]
        _hold(got[np.ix_(p, c)], xv[p], wv[e][c], K + K // 128, "expert %d" % e)


def _spread(rng, T, K):
    """Numbers of all sizes between 2^-8 and 2^8 around a mean: their sums are not exact."""
    return rng.standard_normal((T, K)) * 2.0 ** rng.integers(-8, 8, (T, K)) + 37.0


@pytest.mark.parametrize("T,N,K", INT4_LINEAR)
def test_int4_weights_of_zero_add_nothing(T, N, K):
    rng = np.random.default_rng(N)
    x = _bf(_spread(rng, T, K))[0]
    w, s, _ = _int4(rng, (N, K), np.full((N, K), 8))
    y = torch.full((T, N), GUARD, device=DEV)
    pe.linear_w4(x, w, s, y)
    torch.cuda.synchronize()
    assert not y.any()


@pytest.mark.parametrize("T,I,H", INT4_GLU)
def test_int4_gates_of_zero_add_nothing(T, I, H):
    """Gates, or up values, whose weights are all zero: every result is zero."""
    rng = np.random.default_rng(I)
    x = _bf(_spread(rng, T, H))[0]
    for half in (slice(0, I), slice(I, 2 * I)):
        codes = rng.integers(0, 16, (2 * I, H))
        codes[half] = 8
        w, s, _ = _int4(rng, (2 * I, H), codes)
        h = torch.full((T, I), GUARD, dtype=torch.bfloat16, device=DEV)
        pe.glu_w4(x, w, s, h)
        torch.cuda.synchronize()
        assert not h.any()


@pytest.mark.parametrize("T,N,K", INT4_LINEAR)
def test_int4_product_of_a_single_weight_is_exact(T, N, K):
    rng = np.random.default_rng(K + N)
    x, xv = _bf(_spread(rng, T, K))
    codes = np.full((N, K), 8)
    at = rng.integers(0, K, N)
    codes[np.arange(N), at] = rng.integers(0, 16, N)
    w, s, wv = _int4(rng, (N, K), codes)
    y = torch.empty((T, N), device=DEV)
    pe.linear_w4(x, w, s, y)
    torch.cuda.synchronize()
    assert np.array_equal(y.cpu().numpy().astype(np.float64), xv[:, at] * wv[np.arange(N), at])


@pytest.mark.parametrize("E,R,N,K", INT4_GROUPED)
def test_grouped_int4_product_of_a_single_weight_is_exact(E, R, N, K):
    rng = np.random.default_rng(K + N)
    offsets = _uneven(rng, E, R)
    x, xv = _bf(_spread(rng, R, K))
    codes = np.full((E, N, K), 8)
    at = rng.integers(0, K, (E, N))
    np.put_along_axis(codes, at[:, :, None], rng.integers(0, 16, (E, N, 1)), 2)
    w, s, wv = _int4(rng, (E, N, K), codes)
    y = torch.empty((R, N), device=DEV)
    pe.grouped_linear(x, w, y, _i32(offsets), w_scales=s)
    torch.cuda.synchronize()
    got = y.cpu().numpy().astype(np.float64)
    for e in range(E):
        p = slice(offsets[e], offsets[e + 1])
        assert np.array_equal(got[p], xv[p][:, at[e]] * wv[e][np.arange(N), at[e]]), e


# ------------------------------------------------------------------ MXFP4 tiles whose k is no multiple of 128

@pytest.mark.parametrize("T,N,K", MX_LINEAR)
def test_mxfp4_tiles_of_any_k(T, N, K):
    rng = np.random.default_rng(T + N + K)
    x, xv = _bf(rng.standard_normal((T, K)))
    w, s, wv, size = _weights(rng, "mxfp4", (N, K))
    out, ok = _padded(T, N, torch.float32)
    pe.linear_w4(x, w, s, out)
    torch.cuda.synchronize()
    r, c = _some(rng, T, 80), _some(rng, N, 80)
    _check_linear(out.cpu().numpy().astype(np.float64)[np.ix_(r, c)], xv[r], wv[c], size[c], K, out_eps=U)
    ok()


@pytest.mark.parametrize("T,I,H", MX_GLU)
def test_mxfp4_glu_tiles_of_any_k(T, I, H):
    rng = np.random.default_rng(T + I + H)
    x, xv = _bf(rng.standard_normal((T, H)))
    w, s, wv, size = _weights(rng, "mxfp4", (2 * I, H))
    out, ok = _padded(T, I)
    pe.glu_w4(x, w, s, out)
    torch.cuda.synchronize()
    r, c = _some(rng, T, 80), _some(rng, I, 80)
    both = np.concatenate([c, I + c])
    _check_glu(_np(out)[np.ix_(r, c)], None, xv[r], wv[both], size[both], H, "silu")
    ok()


@pytest.mark.parametrize("E,R,N,K", MX_GROUPED)
@pytest.mark.parametrize("glu", [False, True])
def test_grouped_mxfp4_tiles_of_any_k(E, R, N, K, glu):
    rng = np.random.default_rng(E + R + N + K)
    N, X = N // 2 // 8 * 8 if glu else N, 50
    offsets, rows = _uneven(rng, E, R), rng.integers(0, X, R)
    x, xv = _bf(rng.standard_normal((X, K)))
    w, s, wv, size = _weights(rng, "mxfp4", (E, (2 if glu else 1) * N, K))
    out, ok = _padded(R, N)
    gu = torch.empty((R, 2 * N), dtype=torch.bfloat16, device=DEV) if glu else None
    if glu:
        pe.grouped_glu(x, w, out, _i32(offsets), rows=_i32(rows), w_scales=s, gu=gu)
    else:
        pe.grouped_linear(x, w, out, _i32(offsets), rows=_i32(rows), w_scales=s)
    torch.cuda.synchronize()
    got, c = _np(out), _some(rng, N, 60)
    both = np.concatenate([c, N + c]) if glu else c
    for e, p in _parts(offsets):
        p = p.start + _some(rng, p.stop - p.start, 40)
        if glu:
            _check_glu(got[np.ix_(p, c)], _np(gu)[np.ix_(p, both)], xv[rows[p]], wv[e][both], size[e][both], K, "silu")
        else:
            _check_linear(got[np.ix_(p, c)], xv[rows[p]], wv[e][c], size[e][c], K)
    ok()


# ------------------------------------------------------------------ every code and every scale

def _scaled(rng, wtype, shape):
    """Weights of every code and scale: device codes and scales, values (64 bits, infinite beyond bf16), and for each row
    the k that are not finite.  The last five rows of each matrix have scales at and past the end of the range."""
    K, N = shape[-1], shape[-2]
    codes = rng.integers(0, 16, shape)
    if wtype == "int4":
        per, names = 128, [0x7C00, 0xFC00, 0x7E00, 0x7C00, 0x7BFF]           # infinities, NaN, the largest
        s = rng.integers(0, 2 ** 16, shape[:-1] + (K // per,)).astype(np.uint16)
        s[(s & 0x7C00) == 0x7C00] ^= 0x4000
        s.reshape(-1)[:4] = 0, 1, 0x8000, 0x8001
        value, scale = codes - 8.0, None
    else:
        per, names = 32, [253, 253, 254, 254, 255]
        s = rng.integers(0, 253, shape[:-1] + (K // per,)).astype(np.uint8)
    at = rng.integers(0, K // per, shape[:-2] + (5,))                        # one group of each of these rows
    for m in np.ndindex(*shape[:-2]):
        for i in range(5):
            n, g = N - 5 + i, at[m + (i,)]
            s[m + (n, g)] = names[i]
            own = codes[m + (n,)][g * per:(g + 1) * per]
            if wtype == "mxfp4" and i < 4:                                   # to 3 * 2^126 or 1.5 * 2^127; odd i: and a six
                own[:] = rng.integers(0, 6 if i < 2 else 4, per) + 8 * rng.integers(0, 2, per)
                if i % 2:
                    own[7] = 15 if i == 3 else 7
    if wtype == "int4":
        scale = s.view(np.float16).astype(np.float64)
        dev = torch.from_numpy(s.view(np.float16)).to(DEV)
    else:
        value = formats.e2m1_to_f32(codes.astype(np.uint8)).astype(np.float64)
        scale = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
        dev = torch.from_numpy(s).to(DEV)
    with np.errstate(invalid="ignore"):
        v = value * np.repeat(scale, per, -1)
        bad = ~np.isfinite(np.repeat(scale, per, -1))
    if wtype == "mxfp4":
        v = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)
        bad = ~np.isfinite(v)
    packed = (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)
    return torch.from_numpy(packed).to(DEV), dev, v, bad


def _picked(v, bad, k, wtype):
    """One matrix's products with rows that are zero but for a one at k: its weights there; a NaN where another weight
    (int4: another group's sum, times its scale) is not finite and meets a zero."""
    y, here = v[:, k].T.copy(), bad[:, k].T
    others = bad.sum(1)[None, :] - here.astype(int)
    y[(others > 0) & ~here if wtype == "int4" else others > 0] = np.nan
    return y


def _hold_picked(got, v, bad, k, wtype, what):
    y = _picked(v, bad, k, wtype)
    assert np.array_equal(got, y, equal_nan=True), (what, np.argwhere(~((got == y) | (np.isnan(got) & np.isnan(y))))[:5])


PICKED_LINEAR = [("int4",) + c for c in INT4_LINEAR] + [("mxfp4",) + c for c in [
    (3, 40, 256), (1, 2048, 1152), (16, 6144, 1120), (16, 2048, 1152), (150, 2048, 1120), (500, 2048, 160),
    (2048, 2048, 288), (2300, 4100, 96)]]
PICKED_GROUPED = [("int4",) + c for c in INT4_GROUPED] + [("mxfp4",) + c for c in [
    (4, 9, 40, 1152), (3, 14, 200, 288), (3, 294, 136, 1120), (2, 1100, 3400, 160), (2, 1100, 6704, 96)]]


@pytest.mark.parametrize("wtype,T,N,K", PICKED_LINEAR)
def test_every_code_and_scale_of_one_matrix(wtype, T, N, K):
    rng = np.random.default_rng(T + N + K)
    w, s, v, bad = _scaled(rng, wtype, (N, K))
    k = rng.permutation(np.arange(max(T, K)) % K)[:T]
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    x[torch.arange(T), torch.from_numpy(k)] = 1.0
    y = torch.empty((T, N), device=DEV)
    pe.linear_w4(x, w, s, y)
    torch.cuda.synchronize()
    _hold_picked(y.cpu().numpy().astype(np.float64), v, bad, k, wtype, "linear_w4")


@pytest.mark.parametrize("wtype,E,R,N,K", PICKED_GROUPED)
@pytest.mark.parametrize("glu", [False, True])
def test_every_code_and_scale_of_experts(wtype, E, R, N, K, glu):
    rng = np.random.default_rng(E + R + N + K)
    N = N // 2 // 8 * 8 if glu else N
    offsets = _uneven(rng, E, R)
    w, s, v, bad = _scaled(rng, wtype, (E, (2 if glu else 1) * N, K))
    k = rng.permutation(np.arange(max(R, K)) % K)[:R]
    x = torch.zeros((R, K), dtype=torch.bfloat16, device=DEV)
    x[torch.arange(R), torch.from_numpy(k)] = 1.0
    if glu:
        h, y = (torch.empty((R, n * N), dtype=torch.bfloat16, device=DEV) for n in (1, 2))
        pe.grouped_glu(x, w, h, _i32(offsets), w_scales=s, gu=y)
        v = torch.from_numpy(v).to(torch.bfloat16).double().numpy()         # rounded once; MXFP4 not at all
    else:
        y = torch.empty((R, N), device=DEV)
        pe.grouped_linear(x, w, y, _i32(offsets), w_scales=s)
    torch.cuda.synchronize()
    got = y.double().cpu().numpy()
    for e, p in _parts(offsets):
        _hold_picked(got[p], v[e], bad[e], k[p], wtype, "expert %d" % e)


PICKED_GLU = [(wtype, T, I, H + left) for wtype, left in (("int4", 0), ("mxfp4", -32)) for T, I, H in INT4_GLU]


@pytest.mark.parametrize("wtype,T,I,H", PICKED_GLU)
def test_every_code_and_scale_of_up_values(wtype, T, I, H):
    """Gates of 0.5: every result is silu(0.5) times one weight."""
    rng = np.random.default_rng(T + I + H)
    w, s, v, bad = _scaled(rng, wtype, (2 * I, H))
    w[:I], s[:I] = (0x99, 0.5) if wtype == "int4" else (0x11, 127)
    k = rng.permutation(np.arange(max(T, H)) % H)[:T]
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    x[torch.arange(T), torch.from_numpy(k)] = 1.0
    h = torch.empty((T, I), dtype=torch.bfloat16, device=DEV)
    pe.glu_w4(x, w, s, h)
    torch.cuda.synchronize()
    got, ref = _np(h), _picked(v[I:], bad[I:], k, wtype) * (0.5 / (1 + np.exp(-0.5)))
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin], equal_nan=True)
    _within(got[fin], ref[fin], np.abs(ref[fin]) * (BF + 2 * FN) + 2.0 ** -133)
