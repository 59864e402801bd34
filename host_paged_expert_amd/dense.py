"""The dense operators around a paged MoE layer, on torch tensors.

Each function checks that the tensors match what the library reads and
writes, takes sizes and row strides from them and calls the C entry point of
the same name (include/pe.h says what each computes).  Outputs are passed in;
nothing is allocated.  As everywhere in this package, `stream` is a torch
stream, an int hipStream_t, or None for the null stream.

Matrices are 2-D with contiguous rows (any row stride the C entry point
takes); weights, scales, `gu`, `dgu`, `h` of ffn_backward and weight gradients
are contiguous.  e4m3 codes are torch.float8_e4m3fn or torch.uint8 tensors.
"""
import torch

from . import _binding as b

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_MAX = 2 ** 31 - 1                        # the C entry points' sizes are ints (and bounded below that); ctypes would wrap


def _plain(t, dtype, shape, d):
    """Whether `t` is a contiguous tensor of this type and shape on GPU `d`: the common case, told quickly.  A decode
    step's calls take a few microseconds each, and this is most of what Python adds to them."""
    try:
        return t.shape == shape and t.dtype is dtype and t.get_device() == d and t.is_contiguous()
    except (AttributeError, TypeError):
        return False


def _mat(name, t, dtypes, shape, d, strided=False):
    """Raise unless `t` is a matrix (or vector) of this shape, type and device; its row stride."""
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype not in dtypes or t.get_device() != d:
        raise ValueError("%s must be a %s tensor on cuda:%d (got %s on %s)" % (
            name, " or ".join(str(k) for k in dtypes), d, t.dtype, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.is_contiguous():
        return shape[-1]
    if not strided or len(shape) != 2:
        raise ValueError("%s must be contiguous" % name)
    row, col = t.stride()
    if shape[0] <= 1:                     # the stride of a single row is any number
        row = shape[1]
    if (col != 1 and shape[1] > 1) or row < shape[1]:
        raise ValueError("%s must have contiguous rows that do not overlap (strides %s)" % (name, t.stride()))
    return row


def _ld(name, t, dtype, shape, d):
    """Row stride of a matrix whose rows may lie apart."""
    return shape[1] if _plain(t, dtype, shape, d) else _mat(name, t, dtype, shape, d, True)


def _need(name, t, dtype, shape, d):
    """Address of a contiguous tensor, or of none if it is optional and absent."""
    if not _plain(t, dtype, shape, d):
        _mat(name, t, dtype, shape, d)
    return t.data_ptr()


def _opt(name, t, dtype, shape, d):
    return None if t is None else _need(name, t, dtype, shape, d)


def _left(name, t):
    """Shape and GPU of the operand the others are checked against."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda or t.dim() != 2:
        raise ValueError("%s must be a matrix on the GPU (got shape %s on %s)" % (name, tuple(t.shape), t.device))
    T, C = t.shape
    if T > _MAX or C > _MAX:
        raise ValueError("%s is too large: %s" % (name, tuple(t.shape)))
    return T, C, t.get_device()


def _choice(name, value, table):
    if value not in table:
        raise ValueError("%s must be one of %s, got %r" % (name, ", ".join(sorted(table)), value))
    return table[value]


def rmsnorm(x, weight, eps, out, scales=None, residual=None, sum_out=None, stream=None):
    """out = rms_norm(x + residual) * weight as bf16, or as e4m3 codes with `scales`
    fp32 [T, H/128]; sum_out (optional) = x + residual as bf16."""
    T, H, d = _left("x", x)
    shape = (T, H)
    ldx = _ld("x", x, _BF16, shape, d)
    ldr = lds = 0
    r = s = None
    if residual is not None:
        ldr, r = _ld("residual", residual, _BF16, shape, d), residual.data_ptr()
    if sum_out is not None:
        lds, s = _ld("sum_out", sum_out, _BF16, shape, d), sum_out.data_ptr()
    w = _need("weight", weight, _BF16, (H,), d)
    if scales is None:
        ldy, q = _ld("out", out, _BF16, shape, d), None
    else:
        ldy = H if _plain(out, _E4M3[0], shape, d) else _mat("out", out, _E4M3, shape, d, True)
        q = _need("scales", scales, _F32, (T, H // 128), d)
    return b.check(b.lib().pe_rmsnorm(d, x.data_ptr(), ldx, r, ldr, w, eps, T, H, s, lds, out.data_ptr(), ldy, q,
                                      b.stream_handle(stream)))


def route(logits, topk_ids, topk_w, scoring="softmax", renormalize=True, scale=1.0, stream=None):
    """Top-k ids (int32 [T, k]) and weights (fp32 [T, k]) of fp32 logits [T, E], for PagedMoE.forward."""
    T, E, d = _left("logits", logits)
    ldl = _ld("logits", logits, _F32, (T, E), d)
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids must be a [T, k] tensor")
    k = topk_ids.shape[1]
    if k > _MAX:
        raise ValueError("topk_ids is too large: %s" % (tuple(topk_ids.shape),))
    ids = _need("topk_ids", topk_ids, _I32, (T, k), d)
    w = _need("topk_w", topk_w, _F32, (T, k), d)
    return b.check(b.lib().pe_route(d, logits.data_ptr(), ldl, T, E, k, _choice("scoring", scoring, b.SCORES),
                                    1 if renormalize else 0, scale, ids, w, b.stream_handle(stream)))


def _operands(x, w, x_scales, w_scales, w_rows):
    """Checks of a product's operands: T, K, GPU, weight format, x's row stride, addresses of w and the scales."""
    T, K, d = _left("x", x)
    if x_scales is None and w_scales is None:
        return (T, K, d, b.PE_W_BF16, _ld("x", x, _BF16, (T, K), d), _need("w", w, _BF16, (w_rows, K), d), None, None)
    ld = K if _plain(x, _E4M3[0], (T, K), d) else _mat("x", x, _E4M3, (T, K), d, True)
    if not _plain(w, _E4M3[0], (w_rows, K), d):
        _mat("w", w, _E4M3, (w_rows, K), d)
    return (T, K, d, b.PE_W_FP8_B128, ld, w.data_ptr(), _need("x_scales", x_scales, _F32, (T, K // 128), d),
            _need("w_scales", w_scales, _F32, (-(-w_rows // 128), K // 128), d))


def linear(x, w, out, x_scales=None, w_scales=None, bias=None, act="none", residual=None, stream=None):
    """out = act(x w^T + bias) + residual, bf16 or fp32 by out's type; bf16 operands, or e4m3
    ones with scales per row and 128 columns (x) and per 128 x 128 block (w)."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [N, K] tensor")
    N = w.shape[0]
    if N > _MAX:
        raise ValueError("w is too large: %s" % (tuple(w.shape),))
    T, K, d, wtype, ldx, wp, xs, ws = _operands(x, w, x_scales, w_scales, N)
    bp = _opt("bias", bias, _BF16, (N,), d)
    ldr, r = 0, None
    if residual is not None:
        ldr, r = _ld("residual", residual, _BF16, (T, N), d), residual.data_ptr()
    ytype = b.PE_Y_BF16
    if _plain(out, _BF16, (T, N), d):
        ldy = N
    else:
        ldy = _mat("out", out, (_BF16, _F32), (T, N), d, True)
        if out.dtype is _F32:
            ytype = b.PE_Y_FP32
    return b.check(b.lib().pe_linear(d, wtype, x.data_ptr(), ldx, xs, wp, ws, bp, _choice("act", act, b.ACTS), r, ldr,
                                     T, N, K, out.data_ptr(), ldy, ytype, b.stream_handle(stream)))


def glu(x, w13, out, x_scales=None, w_scales=None, out_scales=None, act="silu", gu=None, stream=None):
    """out = act(x W1^T) * (x W3^T) with w13 = [W1; W3], as bf16, or as e4m3 codes with
    `out_scales` fp32 [T, I/128]; gu (optional, bf16 [T, 2I]) keeps both projections."""
    if not isinstance(out, torch.Tensor) or out.dim() != 2:
        raise ValueError("out must be a [T, I] tensor")
    I = out.shape[1]
    if I > _MAX:
        raise ValueError("out is too large: %s" % (tuple(out.shape),))
    T, H, d, wtype, ldx, wp, xs, ws = _operands(x, w13, x_scales, w_scales, 2 * I)
    if out_scales is None:
        ldh, hs = _ld("out", out, _BF16, (T, I), d), None
    else:
        ldh = I if _plain(out, _E4M3[0], (T, I), d) else _mat("out", out, _E4M3, (T, I), d, True)
        hs = _need("out_scales", out_scales, _F32, (T, I // 128), d)
    return b.check(b.lib().pe_glu(d, wtype, _choice("act", act, b.ACTS), x.data_ptr(), ldx, xs, wp, ws, T, H, I,
                                  out.data_ptr(), ldh, hs, _opt("gu", gu, _BF16, (T, 2 * I), d),
                                  b.stream_handle(stream)))


def ffn_backward(dy, x, gu, w13, w2, dgu, h=None, dx=None, dw13=None, dw2=None, act="silu", stream=None):
    """Gradients of y = glu(x, w13) w2^T for dy: whichever of dx, dw13, dw2 (bf16) are given.
    gu is glu's kept output; dgu [T, 2I] and (with dw2) h [T, I] are written on the way."""
    T, H, d = _left("dy", dy)
    if not isinstance(w2, torch.Tensor) or w2.dim() != 2:
        raise ValueError("w2 must be a [H, I] tensor")
    I = w2.shape[1]
    if I > _MAX:
        raise ValueError("w2 is too large: %s" % (tuple(w2.shape),))
    lddy = _ld("dy", dy, _BF16, (T, H), d)
    ldx = lddx = 0
    xp = dxp = None
    if x is not None:
        ldx, xp = _ld("x", x, _BF16, (T, H), d), x.data_ptr()
    if dx is not None:
        lddx, dxp = _ld("dx", dx, _BF16, (T, H), d), dx.data_ptr()
    return b.check(b.lib().pe_ffn_backward(
        d, _choice("act", act, b.ACTS), dy.data_ptr(), lddy, xp, ldx, _need("gu", gu, _BF16, (T, 2 * I), d),
        _opt("w13", w13, _BF16, (2 * I, H), d), _need("w2", w2, _BF16, (H, I), d),
        T, H, I, _need("dgu", dgu, _BF16, (T, 2 * I), d), _opt("h", h, _BF16, (T, I), d), dxp, lddx,
        _opt("dw13", dw13, _BF16, (2 * I, H), d), _opt("dw2", dw2, _BF16, (H, I), d), b.stream_handle(stream)))
