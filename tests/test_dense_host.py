"""Refusals of the dense operators' C entry points: every one is decided on the
host before anything touches a GPU, so they run here with made-up addresses."""
import pytest

import host_paged_expert_amd as pe

A = [0x10000000 * (i + 1) for i in range(12)]       # addresses far apart, 16-byte aligned


def _norm(**kw):
    d = dict(device=0, x=A[0], ldx=256, residual=A[1], ldr=256, weight=A[2], eps=1e-6, T=4, H=256, sum_out=A[3],
             lds=256, y=A[4], ldy=256, yscale=None)
    d.update(kw)
    return pe.pe_rmsnorm(**d)


def _route(**kw):
    d = dict(device=0, logits=A[0], ldl=64, T=4, num_experts=64, top_k=4, scoring=0, renormalize=1, scale=1.0,
             topk_ids=A[1], topk_w=A[2])
    d.update(kw)
    return pe.pe_route(**d)


def _linear(**kw):
    d = dict(device=0, wtype=0, x=A[0], ldx=256, xscale=None, w=A[1], wscale=None, bias=A[2], act=0, residual=A[3],
             ldr=100, T=4, N=100, K=256, y=A[4], ldy=100, ytype=0)
    d.update(kw)
    return pe.pe_linear(**d)


def _glu(**kw):
    d = dict(device=0, wtype=0, act=1, x=A[0], ldx=256, xscale=None, w13=A[1], s13=None, T=4, hidden=256, inter=128,
             h=A[2], ldh=128, hscale=None, gu=None)
    d.update(kw)
    return pe.pe_glu(**d)


def _back(**kw):
    d = dict(device=0, act=1, dy=A[0], lddy=256, x=A[1], ldx=256, gu=A[2], w13=A[3], w2=A[4], T=4, hidden=256,
             inter=128, dgu=A[5], h=A[6], dx=A[7], lddx=256, dw13=A[8], dw2=A[9])
    d.update(kw)
    return pe.pe_ffn_backward(**d)


FP8 = dict(wtype=1, xscale=A[6], wscale=A[7])
REFUSED = [
    (_norm, dict(x=None)), (_norm, dict(weight=None)), (_norm, dict(y=None)), (_norm, dict(T=-1)), (_norm, dict(H=0)),
    (_norm, dict(H=252, ldx=256)), (_norm, dict(H=200, yscale=A[5])), (_norm, dict(ldx=255)), (_norm, dict(ldx=257)),
    (_norm, dict(x=A[0] + 2)), (_norm, dict(eps=-1.0)), (_norm, dict(eps=float("nan"))), (_norm, dict(device=-1)),
    (_norm, dict(y=A[0] + 512)), (_norm, dict(y=A[3])), (_norm, dict(y=A[0], ldy=512)), (_norm, dict(sum_out=A[2])),
    (_norm, dict(y=A[0], yscale=A[5])), (_norm, dict(yscale=A[4] + 4)), (_norm, dict(H=16384 + 128, ldx=32768, ldr=32768,
                                                                                 lds=32768, ldy=32768)),
    (_norm, dict(ldx=2 ** 31)), (_norm, dict(ldx=2 ** 22)), (_norm, dict(T=2 ** 24)), (_route, dict(T=2 ** 24)),
    (_linear, dict(T=2 ** 24)), (_linear, dict(N=2 ** 22, ldr=2 ** 22, ldy=2 ** 22)), (_glu, dict(T=2 ** 24)),
    (_back, dict(T=2 ** 24)),
    (_route, dict(logits=None)), (_route, dict(topk_ids=None)), (_route, dict(topk_w=None)), (_route, dict(top_k=65)),
    (_route, dict(top_k=0)), (_route, dict(num_experts=1025, ldl=1025)), (_route, dict(scoring=2)),
    (_route, dict(T=-1)), (_route, dict(ldl=63)), (_route, dict(topk_ids=A[0])), (_route, dict(topk_w=A[1] + 16)),
    (_linear, dict(x=None)), (_linear, dict(w=None)), (_linear, dict(y=None)), (_linear, dict(K=100)),
    (_linear, dict(K=0)), (_linear, dict(N=0)), (_linear, dict(T=-1)), (_linear, dict(act=3)), (_linear, dict(ytype=2)),
    (_linear, dict(ldx=260)), (_linear, dict(x=A[0] + 8)), (_linear, dict(w=A[1] + 8)), (_linear, dict(ldy=99)),
    (_linear, dict(xscale=A[6])), (_linear, dict(y=A[0])), (_linear, dict(y=A[1])), (_linear, dict(y=A[3] + 2)),
    (_linear, dict(y=A[3], ldy=128)), (_linear, dict(y=A[3], ytype=1)), (_linear, dict(y=A[4] + 1)),
    (_linear, dict(bias=A[2] + 1)), (_linear, dict(wtype=1, wscale=A[7])), (_linear, dict(wtype=1, xscale=A[6])),
    (_linear, dict(FP8, K=64)), (_linear, dict(FP8, ldx=264)), (_linear, dict(FP8, y=A[6])),
    (_glu, dict(x=None)), (_glu, dict(w13=None)), (_glu, dict(h=None)), (_glu, dict(act=0)), (_glu, dict(inter=100)),
    (_glu, dict(inter=8, hscale=A[5])), (_glu, dict(hidden=100)), (_glu, dict(h=A[0])), (_glu, dict(gu=A[2])),
    (_glu, dict(wtype=1, xscale=A[6], s13=A[7], inter=64)), (_glu, dict(wtype=1, xscale=A[6])), (_glu, dict(s13=A[7])),
    (_glu, dict(ldh=64)), (_glu, dict(gu=A[5] + 2)), (_glu, dict(T=-2)), (_glu, dict(inter=2 ** 30 + 8, ldh=2 ** 30 + 8)),
    (_back, dict(dy=None)), (_back, dict(x=None)), (_back, dict(gu=None)), (_back, dict(w13=None)),
    (_back, dict(w2=None)), (_back, dict(dgu=None)), (_back, dict(h=None)), (_back, dict(dx=None, dw13=None, dw2=None)),
    (_back, dict(act=0)), (_back, dict(hidden=252)), (_back, dict(inter=100)), (_back, dict(dgu=A[2])),
    (_back, dict(dx=A[0])), (_back, dict(dw13=A[3])), (_back, dict(dw2=A[8])), (_back, dict(lddx=100)),
    (_back, dict(T=-1)), (_back, dict(h=A[5] + 1024)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)), ids=lambda i: "%s-%s" % (
    REFUSED[i][0].__name__[1:], "-".join(REFUSED[i][1])))
def test_refused(i):
    fn, kw = REFUSED[i]
    with pytest.raises(pe.PEError) as ei:
        fn(**kw)
    assert ei.value.code == pe.PE_ERR_INVALID_ARG and pe.pe_last_error()


@pytest.mark.parametrize("wtype", [2, 3, 4])
def test_other_formats_are_unsupported(wtype):
    for fn in (_linear, _glu):
        with pytest.raises(pe.PEError) as ei:
            fn(wtype=wtype)
        assert ei.value.code == pe.PE_ERR_UNSUPPORTED


def test_no_tokens_is_a_no_op():
    for fn in (_norm, _route, _linear, _glu):
        assert fn(T=0) == pe.PE_OK
    assert pe.pe_linear(0, 0, None, 256, None, None, None, None, 0, None, 0, 0, 100, 256, None, 100, 0) == pe.PE_OK


def test_tensor_functions_check_their_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        pe.rmsnorm(x, x[0], 1e-6, x)
    with pytest.raises(TypeError):
        pe.rmsnorm(None, x[0], 1e-6, x)
    with pytest.raises(ValueError, match="topk_ids|on the GPU"):
        pe.route(x.float(), None, None)
    with pytest.raises(ValueError):
        pe.linear(x, None, x)
    with pytest.raises(AttributeError):
        pe.no_such_function


@pytest.mark.parametrize("kw", [dict(inter=2 ** 30, dw2=None), dict(inter=2 ** 21, dw2=None),
                                dict(hidden=2 ** 22, dw13=None)], ids=str)
def test_backward_of_no_tokens_refuses_sizes_beyond_a_row(kw):
    """The bounds on rows hold although T = 0 leaves most of them unread: 2 * inter rows of dw13 are counted in 32 bits."""
    with pytest.raises(pe.PEError) as ei:
        _back(T=0, **kw)
    assert ei.value.code == pe.PE_ERR_INVALID_ARG


def test_tensor_functions_refuse_sizes_that_would_wrap():
    """2^32 + 4 rows are not 4 rows, nor 2^32 + 8 columns 8: nothing is launched for them."""
    torch = pytest.importorskip("torch")

    class OnGpu(torch.Tensor):                       # sizes of a tensor that nothing has to hold
        is_cuda = True

        def get_device(self):
            return 0

    def t(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta").as_subclass(OnGpu)

    n = 2 ** 32
    for call in (lambda: pe.rmsnorm(t(n + 4, 8), t(8), 1e-6, t(n + 4, 8)),
                 lambda: pe.route(t(n + 4, 8, dtype=torch.float32), t(n + 4, 2, dtype=torch.int32), t(n + 4, 2)),
                 lambda: pe.route(t(4, 8, dtype=torch.float32), t(4, n + 2, dtype=torch.int32), t(4, n + 2)),
                 lambda: pe.linear(t(n + 4, 8), t(16, 8), t(n + 4, 16)),
                 lambda: pe.linear(t(4, 8), t(n + 16, 8), t(4, n + 16)),
                 lambda: pe.glu(t(4, 8), t(2 * n + 16, 8), t(4, n + 8)),
                 lambda: pe.ffn_backward(t(4, 8), None, t(4, 2 * n + 16), None, t(8, n + 8), t(4, 2 * n + 16))):
        with pytest.raises(ValueError, match="too large"):
            call()


@pytest.mark.parametrize("kw", [dict(y=A[0] + 256, ldx=256, ldy=256), dict(y=A[0] + 254, ldx=256, ldy=256),
                                dict(y=A[0] + 512 + 312 + 2, ldx=256, ldy=256),
                                dict(y=A[0] + 256, ldx=256, ldy=512)], ids=str)
def test_column_ranges_that_share_bytes_are_refused(kw):
    """x is columns 0 .. 127 of rows of 256 (the last case: y's rows are as far apart as two of x's), y 100 columns
    of the same rows that begin inside x, or end in the next row's x."""
    d = dict(K=128, N=100, residual=None, bias=None)
    if kw["y"] == A[0] + 256 and kw["ldy"] == 256:
        d["N"], d["ldy"] = 129, 256                  # columns 128 .. 256: one too many
    with pytest.raises(pe.PEError) as ei:
        _linear(**dict(kw, **d))
    assert ei.value.code == pe.PE_ERR_INVALID_ARG and b"overlaps" in pe.pe_last_error().encode()
