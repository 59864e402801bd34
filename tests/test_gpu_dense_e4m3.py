"""What include/pe.h says of e4m3 sums and of special values in a scale group (MI355X only)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import dense
from test_gpu_dense import DEV, _bf, _codes, _dev8, _np

pytestmark = pytest.mark.gpu
ONE, MAX, NEG = 0x38, 0x7E, 0xFE          # 1, 448, -448


@pytest.mark.parametrize("T,N", [(1, 16), (8, 64), (40, 200), (300, 700)])
def test_sums_of_cancelling_products(T, N):
    """448 * 448 - 448 * 448 + 1 in one group of eight k: exact with an fp32 output; with a bf16 one off by at most
    7 * 2^-13 of the largest product.  In different groups of eight nothing is lost."""
    x, w = np.zeros((T, 256), np.uint8), np.zeros((N, 256), np.uint8)
    x[:, 128:131], w[:, 128:131] = [MAX, MAX, ONE], [MAX, NEG, ONE]
    apart_x, apart_w = np.zeros_like(x), np.zeros_like(w)
    apart_x[:, [0, 8, 16]], apart_w[:, [0, 8, 16]] = [MAX, MAX, ONE], [MAX, NEG, ONE]
    s = dict(x_scales=torch.ones((T, 2), device=DEV), w_scales=torch.ones((-(-N // 128), 2), device=DEV))
    y32, y16 = torch.zeros((T, N), device=DEV), torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    pe.linear(_dev8(x), _dev8(w), y32, **s)
    pe.linear(_dev8(x), _dev8(w), y16, **s)
    torch.cuda.synchronize()
    assert bool((y32 == 1).all())
    assert float((y16.float() - 1).abs().max()) <= 7 * 2.0 ** -13 * 448 ** 2
    pe.linear(_dev8(apart_x), _dev8(apart_w), y32, **s)
    torch.cuda.synchronize()
    assert bool((y32 == 1).all())


@pytest.mark.parametrize("T", [1, 20, 300])
def test_a_nan_and_an_infinity_in_a_scale_group(T):
    """A column that is NaN is a NaN code in a group whose scale is the others'; a group with an infinity reads back as
    NaN; the groups beside them are as without."""
    rng = np.random.default_rng(T)
    H, I = 256, 512
    x, _ = _bf(rng.standard_normal((T, H)))
    w, _ = _bf(rng.standard_normal((2 * I, H)) * 0.1)

    def run(w):
        h, s = torch.zeros((T, I), dtype=torch.float8_e4m3fn, device=DEV), torch.zeros((T, I // 128), device=DEV)
        pe.glu(x, w, h, out_scales=s)
        torch.cuda.synchronize()
        return _codes(h), _np(s)
    x[:, 0] = x[:, 0].abs() + 1
    w[:, 0], w[5] = 0, 0                              # g = 0: h = 0 in column 5, so that it has no part in the scale
    base, base_s = run(w)
    w[5] = float("nan")
    got, got_s = run(w)
    assert (got[:, 5] & 0x7F == 0x7F).all() and (got_s == base_s).all()
    keep = np.arange(I) != 5
    assert (got[:, keep] == base[:, keep]).all()
    w[5] = 0
    w[200, 0] = float("inf")                          # g = +infinity, u finite and not zero: h is an infinity
    got, got_s = run(w)
    with np.errstate(invalid="ignore"):
        v = dense.dequant_rows(got, got_s)
    assert np.isinf(got_s[:, 1]).all() and np.isnan(v[:, 128:256]).all()
    keep = np.r_[0:128, 256:512]
    assert (got[:, keep] == base[:, keep]).all() and (got_s[:, [0, 2, 3]] == base_s[:, [0, 2, 3]]).all()
