"""RMS norm of rows whose squares pass fp32's range, up to rows full of bf16's largest number (MI355X only)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import dense
from test_gpu_dense import BF, DEV, F8, _bf, _codes, _np, _within

pytestmark = pytest.mark.gpu
LARGEST = float(torch.finfo(torch.bfloat16).max)


def _tol(y, H):
    # as for ordinary rows (half of the sum's relative error, (H / 2) 2^-24, through the root; the root, the
    # division and the products), two more products for the scaling by 2^-75, which is exact where it stays in
    # range; an element below 2^-126 of the row's largest is lost, which is less than 2^-100 of y
    return np.abs(y) * (BF + (H / 2 + 20) * 2.0 ** -24) + 2.0 ** -80


@pytest.mark.parametrize("H", [1024, 4096, 4136, 8192, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_full_of_the_largest_numbers(H, residual):
    """Every element's square passes the range, and so would the sum of all under too weak a scaling."""
    rng = np.random.default_rng(H)
    sign = rng.integers(0, 2, (5, H)) * 2.0 - 1
    a = sign * LARGEST
    a[1] = rng.standard_normal(H)
    a[3] = sign[3] * 2.0 ** 64
    if residual:                                    # half in each: their sum is exact
        a[[0, 2, 4]] /= 2
    x, xv = _bf(a)
    r, rv = _bf(a * (np.arange(5) % 2 == 0)[:, None]) if residual else (None, None)
    w, wv = _bf(1 + 0.1 * rng.standard_normal(H))
    v, y = dense.rmsnorm(xv, rv, wv, 1e-6)
    out, s = torch.zeros_like(x), torch.zeros_like(x)
    pe.rmsnorm(x, w, 1e-6, out, residual=r, sum_out=s)
    torch.cuda.synchronize()
    _within(_np(out), y, _tol(y, H), "y")
    assert (_np(s) == v).all()
    if H % 128 == 0:
        codes = torch.zeros((5, H), dtype=torch.float8_e4m3fn, device=DEV)
        sc = torch.zeros((5, H // 128), device=DEV)
        pe.rmsnorm(x, w, 1e-6, codes, scales=sc, residual=r)
        torch.cuda.synchronize()
        rel = (H / 2 + 20) * 2.0 ** -24
        got = dense.dequant_rows(_codes(codes), _np(sc))
        _within(got, y, np.abs(y) * (F8 * (1 + rel) + rel) + np.repeat(_np(sc), 128, 1) * 2.0 ** -9.9, "codes")


@pytest.mark.parametrize("H", [256, 8192, 16384])
def test_an_eps_as_large_as_the_squares_counts(H):
    """eps may be any number: beside squares of 2^122 one of 2^121 is half of them, and one of 1e-6 nothing; one near
    fp32's largest passes the range only with the mean of the squares."""
    a = np.full((3, H), 2.0 ** 61)
    a[1] = 2.0 ** 58
    a[2] = 1.5 * 2.0 ** 59
    x, xv = _bf(a)
    w, wv = _bf(np.ones(H))
    for eps in (3.4e38, 2.0 ** 121, 2.0 ** 115, 1e-6):
        _, y = dense.rmsnorm(xv, None, wv, eps)
        out = torch.zeros_like(x)
        pe.rmsnorm(x, w, eps, out)
        torch.cuda.synchronize()
        _within(_np(out), y, _tol(y, H), "eps %g" % eps)
