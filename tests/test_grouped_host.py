"""Refusals of the 4-bit and of the expert-grouped operators' C entry points: every one is decided on the host before
anything touches a GPU, so they run here with made-up addresses; and the oracle of the grouped operators against plain
loops."""
import numpy as np
import pytest

import host_paged_expert_amd as pe
from oracle import dense, grouped

A = [0x10000000000 * (i + 1) for i in range(12)]       # addresses far apart, 16-byte aligned
INT4, MX = pe.PE_W_INT4_G128, pe.PE_W_MXFP4_B32


def _call(fn, defaults, kw):
    d = dict(defaults)
    d.update(kw)
    return fn(**d)


def _lin4(**kw):
    return _call(pe.pe_linear_w4, dict(
        device=0, wtype=INT4, x=A[0], ldx=256, w=A[1], wscale=A[2], bias=A[3], act=0, residual=A[4], ldr=100, T=4, N=100,
        K=256, y=A[5], ldy=100, ytype=0), kw)


def _glu4(**kw):
    return _call(pe.pe_glu_w4, dict(device=0, wtype=MX, act=1, x=A[0], ldx=256, w13=A[1], s13=A[2], T=4, hidden=256,
                                    inter=64, h=A[3], ldh=64), kw)


def _rows(**kw):
    return _call(pe.pe_group_rows, dict(device=0, topk_ids=A[0], T=4, top_k=2, num_experts=8, offsets=A[1], rows=A[2],
                                        places=A[3]), kw)


def _glin(**kw):
    return _call(pe.pe_grouped_linear, dict(
        device=0, wtype=0, x=A[0], ldx=256, x_rows=10, rows=A[1], offsets=A[2], w=A[3], wscale=None, bias=A[5], act=0, R=20,
        num_experts=8, N=100, K=256, y=A[6], ldy=100, ytype=0), kw)


def _gglu(**kw):
    return _call(pe.pe_grouped_glu, dict(
        device=0, wtype=0, act=1, x=A[0], ldx=256, x_rows=10, rows=A[1], offsets=A[2], w13=A[3], s13=None, R=20,
        num_experts=8, hidden=256, inter=64, h=A[5], ldh=64, gu=A[6]), kw)


def _comb(**kw):
    return _call(pe.pe_combine, dict(device=0, y=A[0], ldy=64, R=20, places=A[1], topk_w=A[2], residual=A[3], ldr=64, T=4,
                                     top_k=2, H=64, out=A[4], ldo=64), kw)


def _cback(**kw):
    return _call(pe.pe_combine_backward, dict(
        device=0, dout=A[0], lddo=64, places=A[1], topk_w=A[2], y=A[3], ldy=64, R=20, T=4, top_k=2, H=64, dy=A[4], lddy=64,
        dtopk_w=A[5]), kw)


def _gback(**kw):
    return _call(pe.pe_grouped_ffn_backward, dict(
        device=0, act=1, dy=A[0], lddy=256, x=A[1], ldx=256, x_rows=10, rows=A[2], offsets=A[3], gu=A[4], w13=A[5], w2=A[6],
        R=20, num_experts=8, hidden=256, inter=64, dgu=A[7], h=A[8], dx=A[9], lddx=256, dw13=A[10], dw2=A[11]), kw)


REFUSED = [
    (_lin4, dict(x=None)), (_lin4, dict(w=None)), (_lin4, dict(wscale=None)), (_lin4, dict(y=None)), (_lin4, dict(K=192)),
    (_lin4, dict(wtype=MX, K=144)), (_lin4, dict(K=0)), (_lin4, dict(N=0)), (_lin4, dict(T=-1)), (_lin4, dict(act=3)),
    (_lin4, dict(ytype=2)), (_lin4, dict(ldx=260)), (_lin4, dict(ldx=128)), (_lin4, dict(x=A[0] + 8)),
    (_lin4, dict(w=A[1] + 8)), (_lin4, dict(wscale=A[2] + 2)), (_lin4, dict(ldy=99)), (_lin4, dict(y=A[0])),
    (_lin4, dict(y=A[1] + 64)), (_lin4, dict(y=A[2])), (_lin4, dict(y=A[4] + 2)), (_lin4, dict(y=A[5] + 1)),
    (_lin4, dict(bias=A[3] + 1)), (_lin4, dict(device=-1)), (_lin4, dict(T=2 ** 24)), (_lin4, dict(N=2 ** 22, ldy=2 ** 22)),
    (_lin4, dict(T=2 ** 23, N=2 ** 20, ldy=2 ** 20, ldr=2 ** 20)), (_lin4, dict(ldy=2 ** 22)),
    (_glu4, dict(x=None)), (_glu4, dict(w13=None)), (_glu4, dict(s13=None)), (_glu4, dict(h=None)), (_glu4, dict(act=0)),
    (_glu4, dict(inter=60)), (_glu4, dict(hidden=240)), (_glu4, dict(h=A[0])), (_glu4, dict(h=A[1])), (_glu4, dict(ldh=60)),
    (_glu4, dict(T=-2)), (_glu4, dict(hidden=2 ** 22, ldx=2 ** 22)),
    (_rows, dict(topk_ids=None)), (_rows, dict(offsets=None)), (_rows, dict(rows=None)), (_rows, dict(places=None)),
    (_rows, dict(top_k=0)), (_rows, dict(num_experts=0)), (_rows, dict(num_experts=1025)), (_rows, dict(T=-1)),
    (_rows, dict(T=2 ** 23, top_k=2)), (_rows, dict(places=A[0])), (_rows, dict(rows=A[3] + 4)), (_rows, dict(offsets=A[2])),
    (_rows, dict(rows=A[2] + 2)), (_rows, dict(T=0, offsets=None)),
    (_glin, dict(x=None)), (_glin, dict(w=None)), (_glin, dict(offsets=None)), (_glin, dict(y=None)), (_glin, dict(x_rows=0)),
    (_glin, dict(x_rows=2 ** 24)), (_glin, dict(wscale=A[4])), (_glin, dict(wtype=INT4)), (_glin, dict(K=252)),
    (_glin, dict(wtype=MX, wscale=A[4], K=240)), (_glin, dict(R=-1)), (_glin, dict(num_experts=0)),
    (_glin, dict(num_experts=1025)), (_glin, dict(y=A[0])), (_glin, dict(y=A[1])), (_glin, dict(y=A[2])),
    (_glin, dict(y=A[3])), (_glin, dict(y=A[5])), (_glin, dict(wtype=INT4, wscale=A[4], y=A[4])), (_glin, dict(rows=A[1] + 2)),
    (_glin, dict(offsets=A[2] + 1)), (_glin, dict(ldx=200)), (_glin, dict(act=9)), (_glin, dict(ytype=5)),
    (_glin, dict(rows=None, ldx=2 ** 22)), (_glin, dict(R=2 ** 23, N=2 ** 20, ldy=2 ** 20)),
    (_gglu, dict(x=None)), (_gglu, dict(w13=None)), (_gglu, dict(h=None)), (_gglu, dict(offsets=None)), (_gglu, dict(act=0)),
    (_gglu, dict(inter=60)), (_gglu, dict(gu=A[6] + 2)), (_gglu, dict(gu=A[5])), (_gglu, dict(gu=A[0])), (_gglu, dict(h=A[1])),
    (_gglu, dict(h=A[3] + 64)), (_gglu, dict(s13=A[4])), (_gglu, dict(wtype=MX)), (_gglu, dict(R=2 ** 24)),
    (_comb, dict(y=None)), (_comb, dict(places=None)), (_comb, dict(out=None)), (_comb, dict(H=60)), (_comb, dict(top_k=0)),
    (_comb, dict(R=-1)), (_comb, dict(out=A[0])), (_comb, dict(out=A[3] + 16)), (_comb, dict(out=A[1])), (_comb, dict(ldy=60)),
    (_comb, dict(y=A[0] + 8)), (_comb, dict(places=A[1] + 2)), (_comb, dict(topk_w=A[2] + 1)), (_comb, dict(T=2 ** 23, top_k=512)),
    (_comb, dict(out=A[3], ldo=72)),
    (_cback, dict(dout=None)), (_cback, dict(places=None)), (_cback, dict(y=None)), (_cback, dict(dy=None, dtopk_w=None)),
    (_cback, dict(dy=A[0])), (_cback, dict(dy=A[3])), (_cback, dict(dtopk_w=A[2])), (_cback, dict(dtopk_w=A[4])),
    (_cback, dict(H=12)), (_cback, dict(lddy=60)), (_cback, dict(dtopk_w=A[5] + 2)), (_cback, dict(T=2 ** 22, top_k=16)),
    (_cback, dict(R=2 ** 24)),
    (_gback, dict(dy=None)), (_gback, dict(x=None)), (_gback, dict(gu=None)), (_gback, dict(w13=None)), (_gback, dict(w2=None)),
    (_gback, dict(dgu=None)), (_gback, dict(h=None)), (_gback, dict(offsets=None)), (_gback, dict(dx=None, dw13=None, dw2=None)),
    (_gback, dict(act=0)), (_gback, dict(hidden=252)), (_gback, dict(inter=60)), (_gback, dict(dgu=A[4])), (_gback, dict(dx=A[0])),
    (_gback, dict(dw13=A[5])), (_gback, dict(dw2=A[10])), (_gback, dict(lddx=100)), (_gback, dict(R=-1)), (_gback, dict(x_rows=0)),
    (_gback, dict(dgu=A[2])), (_gback, dict(h=A[3])), (_gback, dict(num_experts=1025)), (_gback, dict(rows=A[2] + 1)),
    (_gback, dict(inter=2 ** 21)), (_gback, dict(hidden=2 ** 22)), (_gback, dict(R=0, offsets=None)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)), ids=lambda i: "%s-%s" % (
    REFUSED[i][0].__name__[1:], "-".join(REFUSED[i][1])))
def test_refused(i):
    fn, kw = REFUSED[i]
    with pytest.raises(pe.PEError) as ei:
        fn(**kw)
    assert ei.value.code == pe.PE_ERR_INVALID_ARG and pe.pe_last_error()


@pytest.mark.parametrize("fn,wtypes", [(_lin4, (0, 1, 3, 5)), (_glu4, (0, 1, 3, -1)), (_glin, (1, 3, 5)), (_gglu, (1, 3, 99))])
def test_other_formats_are_unsupported(fn, wtypes):
    for wtype in wtypes:
        with pytest.raises(pe.PEError) as ei:
            fn(wtype=wtype)
        assert ei.value.code == pe.PE_ERR_UNSUPPORTED


def test_nothing_to_do():
    for fn in (_lin4, _glu4, _comb, _cback):
        assert fn(T=0) == pe.PE_OK
    for fn in (_glin, _gglu):
        assert fn(R=0) == pe.PE_OK


def test_oracle_of_the_grouped_operators():
    """Offsets, rows and places belong together, a grouped product is each row's own, and combine_backward's gradients
    are the differences of combine."""
    rng = np.random.default_rng(0)
    T, k, E, H, N = 9, 3, 5, 6, 4
    ids = rng.integers(-1, E + 1, (T, k))
    offsets, rows, places = grouped.group_rows(ids, E)
    assert offsets[0] == 0 and offsets[-1] == len(rows) == ((ids >= 0) & (ids < E)).sum()
    for t in range(T):
        for j in range(k):
            p, e = places[t, j], ids[t, j]
            assert (p == -1) == (not 0 <= e < E)
            if p >= 0:
                assert rows[p] == t and offsets[e] <= p < offsets[e + 1]
    assert all(np.all(np.diff(rows[offsets[e]:offsets[e + 1]]) >= 0) for e in range(E))
    x, w, b = rng.standard_normal((T, H)), rng.standard_normal((E, N, H)), rng.standard_normal((E, N))
    y = grouped.linear(x, w, b, "silu", offsets, rows, len(rows) + 2)
    assert np.isnan(y[len(rows):]).all()
    for t in range(T):
        for j in range(k):
            if places[t, j] >= 0:
                e = ids[t, j]
                assert np.allclose(y[places[t, j]], dense.act(w[e] @ x[t] + b[e], "silu"), rtol=1e-12)
    y, wt, dout = y[:len(rows)], rng.standard_normal((T, k)), rng.standard_normal((T, N))
    dy, dw = grouped.combine_backward(dout, places, wt, y)

    def loss(y, wt):
        return float((grouped.combine(y, places, wt, None) * dout).sum())
    for arr, grad, at in [(y, dy, p) for p in np.ndindex(y.shape)] + [(wt, dw, p) for p in np.ndindex(wt.shape)]:
        keep = arr[at]
        arr[at] = keep + 0.5
        up = loss(y, wt)
        arr[at] = keep - 0.5
        down = loss(y, wt)
        arr[at] = keep
        assert abs(up - down - grad[at]) < 1e-9                  # combine is linear in each
