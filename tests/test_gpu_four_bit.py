"""The 4-bit products at the ends of their inputs' ranges, in the kernels of few rows and in every tile (MI355X only).

The shapes say which kernel a call takes; test_four_bit_launches.py holds them to it.  An int4 product adds up
x (q - 8) / 16, each term exact, 128 of them at a time, and those sums times 16 s (exact in fp32): an fp32 result is off by
at most (K + K / 128 + 8) * 2^-24 * sum |x (q - 8) s|, and a single weight's product (8 + 4 + 11 bits) not at all.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import formats
from test_gpu_dense import BF, DEV, GUARD, _bf, _np, _within
from test_gpu_grouped import U, _i32, _some, _uneven

pytestmark = pytest.mark.gpu

# (rows, columns, k) of linear_w4
INT4_LINEAR = [(3, 40, 256), (1, 2048, 1152), (16, 6144, 1152), (16, 2048, 1152), (150, 2048, 1152), (500, 2048, 256),
               (2048, 2048, 256), (2300, 4100, 256)]
# (rows, columns, k) of glu_w4
INT4_GLU = [(5, 24, 256), (9, 768, 1152), (8, 8208, 256), (150, 1088, 1152), (500, 1024, 256), (2048, 1024, 256),
            (2300, 2056, 256)]
# (experts, rows, columns, k) of the grouped products
INT4_GROUPED = [(4, 9, 40, 1152), (3, 14, 200, 256), (3, 294, 136, 1152), (2, 1100, 3400, 256), (2, 1100, 6704, 256)]


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
