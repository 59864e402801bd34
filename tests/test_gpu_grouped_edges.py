"""Calls at the edges of the expert-grouped operators (MI355X only)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import host_paged_expert_amd as pe
from oracle import grouped
from test_gpu_dense import BF, DEV, GUARD, _bf, _np, _within
from test_gpu_grouped import U, _check_glu, _check_linear, _i32, _some, _terms, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward_of_tokens_without_rows(weighted):
    """Every id names an expert that is elsewhere: no rows here, tokens all the same."""
    T, k, H = 5, 3, 64
    bf = dict(dtype=torch.bfloat16, device=DEV)
    dout, none = torch.ones((T, H), **bf), torch.empty((0, H), **bf)
    places = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    w = torch.ones((T, k), device=DEV) if weighted else None
    pe.combine_backward(dout, places, none, topk_w=w)
    dw = torch.full((T, k), GUARD, device=DEV)
    pe.combine_backward(dout, places, none, topk_w=w, y=none, dtopk_w=dw)
    torch.cuda.synchronize()
    assert not dw.any()


def test_places_named_twice():
    """combine adds a row as often as it is named; combine_backward without dy gives each entry its own product."""
    T, k, H = 6, 4, 264
    rng = np.random.default_rng(3)
    y, yv = _bf(rng.standard_normal((5, H)))
    dout, dv = _bf(rng.standard_normal((T, H)))
    places = rng.integers(0, 5, (T, k)).astype(np.int32)
    places[0] = 2
    w = rng.standard_normal((T, k)).astype(np.float32)
    out, dw = torch.empty((T, H), dtype=torch.bfloat16, device=DEV), torch.full((T, k), GUARD, device=DEV)
    pe.combine(y, _i32(places), out, topk_w=torch.from_numpy(w).to(DEV))
    pe.combine_backward(dout, _i32(places), y=y, dtopk_w=dw)
    torch.cuda.synchronize()
    ref, size = (grouped.combine(v, places, a.astype(np.float64), None) for v, a in ((yv, w), (np.abs(yv), np.abs(w))))
    _within(_np(out), ref, BF * np.abs(ref) + size * (k + 2) * U * (1 + BF) + 1e-30)
    _, ref = grouped.combine_backward(dv, places, None, yv)
    _, size = grouped.combine_backward(np.abs(dv), places, None, np.abs(yv))
    _within(dw.cpu().numpy().astype(np.float64), ref, size * (H + 8) * U + 1e-30)


@pytest.mark.parametrize("wtype", ["int4", "mxfp4"])
def test_4bit_weights_past_32_bits(wtype):
    """The last of many experts, and the last rows of one large matrix, behind 2^31 bytes of codes."""
    rng = np.random.default_rng(4)
    E, N, K = 530, 1024, 8192                                    # 2.2e9 bytes
    zero = 0x88 if wtype == "int4" else 0
    w = torch.full((E, N, K // 2), zero, dtype=torch.uint8, device=DEV)
    last, ls, lv, size = _weights(rng, wtype, (N, K))
    s = torch.ones((E,) + ls.shape, dtype=ls.dtype, device=DEV)
    w[E - 1], s[E - 1] = last, ls
    x, xv = _bf(rng.standard_normal((8, K)))
    c = _some(rng, N // 2, 40)
    both = np.concatenate([c, N // 2 + c])
    for R in (3, 9000):                                          # under 4 rows an expert, and 16 and more: tiles
        o = np.full(E + 1, R - 2, np.int32)
        o[0], o[E] = 0, R
        rows = rng.integers(0, 8, R).astype(np.int32)
        y, h = (torch.full((R, n), GUARD, dtype=torch.bfloat16, device=DEV) for n in (N, N // 2))
        pe.grouped_linear(x, w, y, _i32(o), rows=_i32(rows), w_scales=s)
        pe.grouped_glu(x, w, h, _i32(o), rows=_i32(rows), w_scales=s)
        torch.cuda.synchronize()
        xr = xv[rows[R - 2:]]
        _check_linear(_np(y[R - 2:]), xr, lv, size, _terms(wtype, K))
        _check_glu(_np(h[R - 2:])[:, c], None, xr, lv[both], size[both], _terms(wtype, K), "silu")
        assert not y[:R - 2].any() and not h[:R - 2].any()
    w, s = w.view(E * N, K // 2), s.view(E * N, -1)
    for T in (2, 8):
        y = torch.full((T, E * N), GUARD, dtype=torch.bfloat16, device=DEV)
        pe.linear_w4(x[:T], w, s, y)
        torch.cuda.synchronize()
        _check_linear(_np(y[:, -N:]), xv[:T], lv, size, _terms(wtype, K))
        assert not y[:, :-N].any()


@pytest.mark.parametrize("wtype", ["int4", "mxfp4"])
def test_4bit_calls_captured_and_replayed(wtype):
    """Two graphs of the same calls on streams of their own, replayed at once on new inputs and other experts' rows, against
    eager calls: streaming and tiles."""
    rng = np.random.default_rng(5)
    E, H, I, k = 6, 512, 64, 2
    w13, s13, _, _ = _weights(rng, wtype, (E, 2 * I, H))
    w2, s2, _, _ = _weights(rng, wtype, (E, H, I * 2))           # (k a multiple of 128)
    ws, ss, _, _ = _weights(rng, wtype, (H, H))

    def buffers(T):
        bf, i32, R = dict(dtype=torch.bfloat16, device=DEV), dict(dtype=torch.int32, device=DEV), T * k
        return dict(x=torch.zeros((T, H), **bf), ids=torch.zeros((T, k), **i32), o=torch.zeros(E + 1, **i32),
                    rows=torch.zeros(R, **i32), places=torch.zeros((T, k), **i32), h=torch.zeros((R, I), **bf),
                    h2=torch.zeros((R, 2 * I), **bf), y=torch.zeros((R, H), **bf), out=torch.zeros((T, H), **bf))

    def step(b, stream):
        pe.group_rows(b["ids"], b["o"], b["rows"], b["places"], stream=stream)
        pe.grouped_glu(b["x"], w13, b["h"], b["o"], rows=b["rows"], w_scales=s13, stream=stream)
        pe.grouped_linear(b["h2"], w2, b["y"], b["o"], w_scales=s2, stream=stream)
        pe.combine(b["y"], b["places"], b["out"], residual=b["x"], stream=stream)
        pe.linear_w4(b["out"], ws, ss, b["x"], stream=stream)

    graphs = []
    for T in (5, 300):
        b, side, g = buffers(T), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                step(b, side)
        graphs.append((b, side, g, buffers(T)))
    for _ in range(3):
        for b, side, g, eager in graphs:
            T = b["x"].shape[0]
            new = dict(x=_bf(rng.standard_normal((T, H)))[0], ids=_i32(rng.integers(-1, E, (T, k))),
                       h2=_bf(rng.standard_normal((T * k, 2 * I)))[0])
            for n, v in new.items():
                b[n].copy_(v)
                eager[n].copy_(v)
        torch.cuda.synchronize()
        for _, side, g, _ in graphs:
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for b, _, _, eager in graphs:
            step(eager, torch.cuda.current_stream())
            torch.cuda.synchronize()
            for n in b:
                assert torch.equal(b[n], eager[n]), n
