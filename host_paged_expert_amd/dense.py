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

_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_E4M3 = (torch.float8_e4m3fn, torch.uint8)


def _mat(name, t, dtypes, shape, dev, strided=False):
    """Raise unless `t` is a matrix (or vector) of this shape, type and device; its row stride."""
    try:
        if t.shape == shape and t.dtype in dtypes and t.device == dev and t.is_contiguous():
            return shape[-1]
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype not in dtypes or t.device != dev:
        raise ValueError("%s must be a %s tensor on %s (got %s on %s)" % (
            name, " or ".join(str(d) for d in dtypes), dev, t.dtype, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not strided or len(shape) != 2:
        raise ValueError("%s must be contiguous" % name)
    row, col = t.stride()
    if shape[0] <= 1:                     # the stride of a single row is any number
        row = shape[1]
    if (col != 1 and shape[1] > 1) or row < shape[1]:
        raise ValueError("%s must have contiguous rows that do not overlap (strides %s)" % (name, t.stride()))
    return row


def _left(name, t):
    """Shape and device of the operand the others are checked against."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dim() != 2 or t.device.type != "cuda":
        raise ValueError("%s must be a matrix on the GPU (got shape %s on %s)" % (name, tuple(t.shape), t.device))
    return t.shape[0], t.shape[1], t.device


def _opt(name, t, dtypes, shape, dev, strided=False):
    return 0 if t is None else _mat(name, t, dtypes, shape, dev, strided)


def _choice(name, value, table):
    if value not in table:
        raise ValueError("%s must be one of %s, got %r" % (name, ", ".join(sorted(table)), value))
    return table[value]


def rmsnorm(x, weight, eps, out, scales=None, residual=None, sum_out=None, stream=None):
    """out = rms_norm(x + residual) * weight as bf16, or as e4m3 codes with `scales`
    fp32 [T, H/128]; sum_out (optional) = x + residual as bf16."""
    T, H, dev = _left("x", x)
    ldx = _mat("x", x, _BF16, (T, H), dev, True)
    _mat("weight", weight, _BF16, (H,), dev)
    ldr = _opt("residual", residual, _BF16, (T, H), dev, True)
    lds = _opt("sum_out", sum_out, _BF16, (T, H), dev, True)
    ldy = _mat("out", out, _BF16 if scales is None else _E4M3, (T, H), dev, True)
    _opt("scales", scales, _F32, (T, H // 128), dev)
    return b.pe_rmsnorm(dev.index, x, ldx, residual, ldr, weight, eps, T, H, sum_out, lds, out, ldy, scales, stream)


def route(logits, topk_ids, topk_w, scoring="softmax", renormalize=True, scale=1.0, stream=None):
    """Top-k ids (int32 [T, k]) and weights (fp32 [T, k]) of fp32 logits [T, E], for PagedMoE.forward."""
    T, E, dev = _left("logits", logits)
    ldl = _mat("logits", logits, _F32, (T, E), dev, True)
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids must be a [T, k] tensor")
    k = topk_ids.shape[1]
    _mat("topk_ids", topk_ids, _I32, (T, k), dev)
    _mat("topk_w", topk_w, _F32, (T, k), dev)
    return b.pe_route(dev.index, logits, ldl, T, E, k, _choice("scoring", scoring, b.SCORES), renormalize, scale,
                      topk_ids, topk_w, stream)


def _operands(x, w, x_scales, w_scales, w_rows):
    """Checks of a product's operands: (T, K, device, weight format, x's row stride)."""
    T, K, dev = _left("x", x)
    fp8 = x_scales is not None or w_scales is not None
    ld = _mat("x", x, _E4M3 if fp8 else _BF16, (T, K), dev, True)
    _mat("w", w, _E4M3 if fp8 else _BF16, (w_rows, K), dev)
    if fp8:
        _mat("x_scales", x_scales, _F32, (T, K // 128), dev)
        _mat("w_scales", w_scales, _F32, (-(-w_rows // 128), K // 128), dev)
    return T, K, dev, b.PE_W_FP8_B128 if fp8 else b.PE_W_BF16, ld


def linear(x, w, out, x_scales=None, w_scales=None, bias=None, act="none", residual=None, stream=None):
    """out = act(x w^T + bias) + residual, bf16 or fp32 by out's type; bf16 operands, or e4m3
    ones with scales per row and 128 columns (x) and per 128 x 128 block (w)."""
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [N, K] tensor")
    N = w.shape[0]
    T, K, dev, wtype, ldx = _operands(x, w, x_scales, w_scales, N)
    _opt("bias", bias, _BF16, (N,), dev)
    ldr = _opt("residual", residual, _BF16, (T, N), dev, True)
    ldy = _mat("out", out, _BF16 + _F32, (T, N), dev, True)
    return b.pe_linear(dev.index, wtype, x, ldx, x_scales, w, w_scales, bias, _choice("act", act, b.ACTS), residual,
                       ldr, T, N, K, out, ldy, b.PE_Y_FP32 if out.dtype is torch.float32 else b.PE_Y_BF16, stream)


def glu(x, w13, out, x_scales=None, w_scales=None, out_scales=None, act="silu", gu=None, stream=None):
    """out = act(x W1^T) * (x W3^T) with w13 = [W1; W3], as bf16, or as e4m3 codes with
    `out_scales` fp32 [T, I/128]; gu (optional, bf16 [T, 2I]) keeps both projections."""
    if not isinstance(out, torch.Tensor) or out.dim() != 2:
        raise ValueError("out must be a [T, I] tensor")
    I = out.shape[1]
    T, H, dev, wtype, ldx = _operands(x, w13, x_scales, w_scales, 2 * I)
    ldh = _mat("out", out, _BF16 if out_scales is None else _E4M3, (T, I), dev, True)
    _opt("out_scales", out_scales, _F32, (T, I // 128), dev)
    _opt("gu", gu, _BF16, (T, 2 * I), dev)
    return b.pe_glu(dev.index, wtype, _choice("act", act, b.ACTS), x, ldx, x_scales, w13, w_scales, T, H, I, out, ldh,
                    out_scales, gu, stream)


def ffn_backward(dy, x, gu, w13, w2, dgu, h=None, dx=None, dw13=None, dw2=None, act="silu", stream=None):
    """Gradients of y = glu(x, w13) w2^T for dy: whichever of dx, dw13, dw2 (bf16) are given.
    gu is glu's kept output; dgu [T, 2I] and (with dw2) h [T, I] are written on the way."""
    T, H, dev = _left("dy", dy)
    if not isinstance(w2, torch.Tensor) or w2.dim() != 2:
        raise ValueError("w2 must be a [H, I] tensor")
    I = w2.shape[1]
    lddy = _mat("dy", dy, _BF16, (T, H), dev, True)
    ldx = _opt("x", x, _BF16, (T, H), dev, True)
    _mat("gu", gu, _BF16, (T, 2 * I), dev)
    _opt("w13", w13, _BF16, (2 * I, H), dev)
    _mat("w2", w2, _BF16, (H, I), dev)
    _mat("dgu", dgu, _BF16, (T, 2 * I), dev)
    _opt("h", h, _BF16, (T, I), dev)
    lddx = _opt("dx", dx, _BF16, (T, H), dev, True)
    _opt("dw13", dw13, _BF16, (2 * I, H), dev)
    _opt("dw2", dw2, _BF16, (H, I), dev)
    return b.pe_ffn_backward(dev.index, _choice("act", act, b.ACTS), dy, lddy, x, ldx, gu, w13, w2, T, H, I, dgu, h, dx,
                             lddx, dw13, dw2, stream)
