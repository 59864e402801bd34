"""The 4-bit products and those grouped by expert, on torch tensors.

As in dense.py each function checks its tensors, takes sizes and row strides from
them and calls the C entry point of the same name (include/pe.h says what each
computes); outputs are passed in, nothing is allocated, and `stream` is a torch
stream, an int hipStream_t, or None for the null stream.

4-bit weights are torch.uint8 with half as many columns, their scales
torch.float16 [..., K/128] (int4) or torch.uint8 [..., K/32] (MXFP4): the scales'
type says which.  Weights and their gradients of E experts are [E, ., .].
Expert e's rows are offsets[e] .. offsets[e+1] - 1 (int32 [E + 1]); rows (int32,
optional) is the row of x that each of them takes.  Rows of the outputs from
offsets[E] on are left as they were.
"""
import torch

from . import _binding as b
from .dense import _BF16, _F32, _I32, _MAX, _choice, _ld, _left, _mat, _need, _opt, _plain

_U8, _F16 = torch.uint8, torch.float16


def _three(name, t):
    """Shape of the weights of several experts."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError("%s must be a [experts, rows, columns] tensor" % name)
    if max(t.shape) > _MAX:
        raise ValueError("%s is too large: %s" % (name, tuple(t.shape)))
    return tuple(t.shape)


def _weights(name, w, scales, shape, d):
    """Format and addresses of weights of this (unpacked) shape and of their scales."""
    if scales is None:
        return b.PE_W_BF16, _need(name, w, _BF16, shape, d), None
    if not isinstance(scales, torch.Tensor):
        raise TypeError("w_scales must be a torch tensor")
    K = shape[-1]
    wtype, dtype, per = (b.PE_W_INT4_G128, _F16, 128) if scales.dtype is _F16 else (b.PE_W_MXFP4_B32, _U8, 32)
    if K % per:
        raise ValueError("%s has %d columns, which are not a multiple of %d" % (name, K, per))
    return (wtype, _need(name, w, _U8, shape[:-1] + (K // 2,), d),
            _need("w_scales", scales, dtype, shape[:-1] + (K // per,), d))


def _out(out, shape, d):
    """Row stride and type of a product's output."""
    if _plain(out, _BF16, shape, d):
        return shape[1], b.PE_Y_BF16
    return _mat("out", out, (_BF16, _F32), shape, d, True), b.PE_Y_FP32 if out.dtype is _F32 else b.PE_Y_BF16


def _row_list(rows, R, d):
    return None if rows is None else _need("rows", rows, _I32, (R,), d)


def linear_w4(x, w, w_scales, out, bias=None, act="none", residual=None, stream=None):
    """out = act(x w^T + bias) + residual, bf16 or fp32 by out's type, for 4-bit weights."""
    T, K, d = _left("x", x)
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] > _MAX:
        raise ValueError("w must be a [N, K/2] tensor")
    N = w.shape[0]
    ldx = _ld("x", x, _BF16, (T, K), d)
    if w_scales is None:
        raise TypeError("w_scales must be a torch tensor")
    wtype, wp, ws = _weights("w", w, w_scales, (N, K), d)
    ldr, r = 0, None
    if residual is not None:
        ldr, r = _ld("residual", residual, _BF16, (T, N), d), residual.data_ptr()
    ldy, ytype = _out(out, (T, N), d)
    return b.check(b.lib().pe_linear_w4(d, wtype, x.data_ptr(), ldx, wp, ws, _opt("bias", bias, _BF16, (N,), d),
                                        _choice("act", act, b.ACTS), r, ldr, T, N, K, out.data_ptr(), ldy, ytype,
                                        b.stream_handle(stream)))


def glu_w4(x, w13, w_scales, out, act="silu", stream=None):
    """out = act(x W1^T) * (x W3^T) as bf16 with w13 = [W1; W3] in 4 bits."""
    T, H, d = _left("x", x)
    if not isinstance(out, torch.Tensor) or out.dim() != 2 or out.shape[1] > _MAX:
        raise ValueError("out must be a [T, I] tensor")
    I = out.shape[1]
    ldx = _ld("x", x, _BF16, (T, H), d)
    if w_scales is None:
        raise TypeError("w_scales must be a torch tensor")
    wtype, wp, ws = _weights("w13", w13, w_scales, (2 * I, H), d)
    return b.check(b.lib().pe_glu_w4(d, wtype, _choice("act", act, b.ACTS), x.data_ptr(), ldx, wp, ws, T, H, I,
                                     out.data_ptr(), _ld("out", out, _BF16, (T, I), d), b.stream_handle(stream)))


def group_rows(topk_ids, offsets, rows, places, stream=None):
    """The routed entries of topk_ids [T, k] in the order of their experts: offsets [E + 1], rows [T * k] (the token of
    each) and places [T, k] (where each entry went, -1 for an id outside [0, E)), all int32."""
    T, k, d = _left("topk_ids", topk_ids)
    ids = _need("topk_ids", topk_ids, _I32, (T, k), d)
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or not 1 <= offsets.shape[0] <= _MAX:
        raise ValueError("offsets must be an [experts + 1] tensor")
    E = offsets.shape[0] - 1
    return b.check(b.lib().pe_group_rows(d, ids, T, k, E, _need("offsets", offsets, _I32, (E + 1,), d),
                                         _need("rows", rows, _I32, (T * k,), d), _need("places", places, _I32, (T, k), d),
                                         b.stream_handle(stream)))


def grouped_linear(x, w, out, offsets, rows=None, w_scales=None, bias=None, act="none", stream=None):
    """out[p] = act(x[rows[p]] w[e]^T + bias[e]) for the rows p of expert e, bf16 or fp32 by out's type; w [E, N, K] bf16,
    or 4-bit with w_scales."""
    X, K, d = _left("x", x)
    E, N, _ = _three("w", w)
    if not isinstance(out, torch.Tensor) or out.dim() != 2 or out.shape[0] > _MAX:
        raise ValueError("out must be a [rows, N] tensor")
    R = out.shape[0]
    if rows is None and X != R:
        raise ValueError("x has %d rows, out %d" % (X, R))
    ldx = _ld("x", x, _BF16, (X, K), d)
    wtype, wp, ws = _weights("w", w, w_scales, (E, N, K), d)
    ldy, ytype = _out(out, (R, N), d)
    return b.check(b.lib().pe_grouped_linear(d, wtype, x.data_ptr(), ldx, X, _row_list(rows, R, d),
                                             _need("offsets", offsets, _I32, (E + 1,), d), wp, ws,
                                             _opt("bias", bias, _BF16, (E, N), d), _choice("act", act, b.ACTS), R, E, N, K,
                                             out.data_ptr(), ldy, ytype, b.stream_handle(stream)))


def grouped_glu(x, w13, out, offsets, rows=None, w_scales=None, act="silu", gu=None, stream=None):
    """out[p] = act(g) * u with g, u = x[rows[p]] w13[e]^T for the rows p of expert e, as bf16; gu (optional, bf16
    [R, 2I]) keeps both.  w13 [E, 2I, H] bf16, or 4-bit with w_scales."""
    X, H, d = _left("x", x)
    E, I2, _ = _three("w13", w13)
    if not isinstance(out, torch.Tensor) or out.dim() != 2 or max(out.shape) > _MAX:
        raise ValueError("out must be a [rows, I] tensor")
    R, I = out.shape
    if rows is None and X != R:
        raise ValueError("x has %d rows, out %d" % (X, R))
    ldx = _ld("x", x, _BF16, (X, H), d)
    wtype, wp, ws = _weights("w13", w13, w_scales, (E, 2 * I, H), d)
    return b.check(b.lib().pe_grouped_glu(d, wtype, _choice("act", act, b.ACTS), x.data_ptr(), ldx, X,
                                          _row_list(rows, R, d), _need("offsets", offsets, _I32, (E + 1,), d), wp, ws, R, E,
                                          H, I, out.data_ptr(), _ld("out", out, _BF16, (R, I), d),
                                          _opt("gu", gu, _BF16, (R, 2 * I), d), b.stream_handle(stream)))


def combine(y, places, out, topk_w=None, residual=None, stream=None):
    """out[t] = sum_j topk_w[t, j] y[places[t, j]] + residual[t] (bf16 [T, H]; without weights they are 1)."""
    R, H, d = _left("y", y)
    if not isinstance(places, torch.Tensor) or places.dim() != 2 or max(places.shape) > _MAX:
        raise ValueError("places must be a [T, k] tensor")
    T, k = places.shape
    ldy = _ld("y", y, _BF16, (R, H), d)
    ldr, r = 0, None
    if residual is not None:
        ldr, r = _ld("residual", residual, _BF16, (T, H), d), residual.data_ptr()
    return b.check(b.lib().pe_combine(d, y.data_ptr(), ldy, R, _need("places", places, _I32, (T, k), d),
                                      _opt("topk_w", topk_w, _F32, (T, k), d), r, ldr, T, k, H, out.data_ptr(),
                                      _ld("out", out, _BF16, (T, H), d), b.stream_handle(stream)))


def combine_backward(dout, places, dy=None, topk_w=None, y=None, dtopk_w=None, stream=None):
    """Gradients of combine for dout [T, H]: dy [R, H] (bf16) and with y dtopk_w [T, k] (fp32), whichever are given."""
    T, H, d = _left("dout", dout)
    if not isinstance(places, torch.Tensor) or places.dim() != 2 or places.shape[1] > _MAX:
        raise ValueError("places must be a [T, k] tensor")
    k = places.shape[1]
    like = dy if dy is not None else y
    if not isinstance(like, torch.Tensor) or like.dim() != 2 or like.shape[0] > _MAX:
        raise ValueError("dy, or y without it, must be a [rows, H] tensor")
    R = like.shape[0]
    ldy = lddy = 0
    yp = dyp = None
    if y is not None:
        ldy, yp = _ld("y", y, _BF16, (R, H), d), y.data_ptr()
    if dy is not None:
        lddy, dyp = _ld("dy", dy, _BF16, (R, H), d), dy.data_ptr()
    return b.check(b.lib().pe_combine_backward(d, dout.data_ptr(), _ld("dout", dout, _BF16, (T, H), d),
                                               _need("places", places, _I32, (T, k), d),
                                               _opt("topk_w", topk_w, _F32, (T, k), d), yp, ldy, R, T, k, H, dyp, lddy,
                                               _opt("dtopk_w", dtopk_w, _F32, (T, k), d), b.stream_handle(stream)))


def grouped_ffn_backward(dy, x, gu, w13, w2, offsets, dgu, rows=None, h=None, dx=None, dw13=None, dw2=None, act="silu",
                         stream=None):
    """Gradients of y = grouped_linear(grouped_glu(x, w13), w2) for dy [R, H]: whichever of dx [R, H] (a row for each of
    y's: `combine` adds up a token's), dw13 and dw2 (bf16) are given.  gu is grouped_glu's kept output; dgu [R, 2I] and
    (with dw2) h [R, I] are written on the way."""
    R, H, d = _left("dy", dy)
    E, _, I = _three("w2", w2)
    lddy = _ld("dy", dy, _BF16, (R, H), d)
    ldx = lddx = X = 0
    xp = dxp = None
    if x is not None:
        X = _left("x", x)[0]
        if rows is None and X != R:
            raise ValueError("x has %d rows, dy %d" % (X, R))
        ldx, xp = _ld("x", x, _BF16, (X, H), d), x.data_ptr()
    if dx is not None:
        lddx, dxp = _ld("dx", dx, _BF16, (R, H), d), dx.data_ptr()
    return b.check(b.lib().pe_grouped_ffn_backward(
        d, _choice("act", act, b.ACTS), dy.data_ptr(), lddy, xp, ldx, X, _row_list(rows, R, d),
        _need("offsets", offsets, _I32, (E + 1,), d), _need("gu", gu, _BF16, (R, 2 * I), d),
        _opt("w13", w13, _BF16, (E, 2 * I, H), d), _need("w2", w2, _BF16, (E, H, I), d), R, E, H, I,
        _need("dgu", dgu, _BF16, (R, 2 * I), d), _opt("h", h, _BF16, (R, I), d), dxp, lddx,
        _opt("dw13", dw13, _BF16, (E, 2 * I, H), d), _opt("dw2", dw2, _BF16, (E, H, I), d), b.stream_handle(stream)))
