"""Binding of include/step.h: the residual's addition with the RMS norm, products
with 4-bit weights, and the choice of the next token (argument marshalling only;
no fallback path).

Tensors are CUDA tensors of the current device; that, shapes, types and strides
are checked here.  Every call enqueues on ``stream`` (default: torch's current
one); on a given stream outputs come from that stream's pool.  Like the package's
other calls they leave no autograd graph."""
from __future__ import annotations

import ctypes

import torch

from . import moe as _moe
from .paged import _check, _i32, _need, _new, _placed, _stream, _used

# names of the functions include/step.h declares (checked by its ABI test)
EXPORTS = ["rms_norm", "linear4", "sample"]

_DTYPE = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3, torch.float8_e4m3fn: 4,
          torch.int8: 5}
_EIGHT = (torch.float8_e4m3fn, torch.int8)
_SCALE = {torch.float16: _moe.MOE_SCALE_F16, torch.bfloat16: _moe.MOE_SCALE_BF16}
_F32 = torch.float32
_lib = None


def _library():
    global _lib
    if _lib is not None:
        return _lib
    lib = _moe.load_library()
    P, I, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    sig = {
        "rms_norm": [P, I, I, I, I, L, L, P, L, L, P, L, L, P, I, I, F, P, I, L, L, P, I, P],
        "linear4": [P, I, I, I, L, P, I, P, P, P, I, I, I, P, I, L, P],
        "sample": [P, I, I, I, L, P, P, P, P, P, F, I, F, F, P, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    _lib = lib
    return lib


def _rows(t, shape, name):
    """Token and head strides of a [T, d] or [T, H, d] tensor whose features are contiguous."""
    if t.shape != shape:
        raise ValueError(f"{name} must be like x")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s features must be contiguous")
    return (st[0], st[1]) if len(st) == 3 else (st[0], 0)


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
             residual: torch.Tensor | None = None, eps: float = 1e-6, unit_offset: bool = False,
             out_dtype: torch.dtype | None = None, group: int = 0,
             out: torch.Tensor | None = None, sum_out: torch.Tensor | None = None, stream=None):
    """RMS norm over the last axis of x [T, d] or [T, H, d] (bf16, fp16 or fp32; any
    strides over the first axes), after the addition of ``residual``; all in fp32.

    ``weight`` [d] of x's type or fp32 (``unit_offset``: 1 + weight).  Returns
    y of ``out_dtype`` (default x's); of torch.float8_e4m3fn or torch.int8: y and its
    scales, fp32 [..., d / group], one for ``group`` features (0: a row); and behind
    them, with a residual, x + residual in x's type.  The last bits of a row may go by how
    many rows the call has (include/step.h).  ``out`` may be x, ``sum_out``
    x or the residual (in place)."""
    shape, xt = x.shape, x.dtype
    dt = _DTYPE.get(xt, 0)
    if not 1 <= dt <= 3 or len(shape) not in (2, 3):
        raise ValueError("x must be [T, d] or [T, H, d] of bf16, fp16 or fp32")
    _placed(x, weight, residual, out, sum_out)
    xs = _rows(x, shape, "x")
    if len(shape) == 2:
        T, d = shape
        H, dense, strides = 1, (d, 1), (d, 0)
    else:
        T, H, d = shape
        dense, strides = (H * d, d, 1), (H * d, d)
    wp = wt = 0
    if weight is not None:
        if weight.dim() != 1 or weight.shape[0] != d or not weight.is_contiguous():
            raise ValueError("weight must be dense [d]")
        wp, wt = weight.data_ptr(), _DTYPE.get(weight.dtype, 0)
    made = []
    if out is None:
        out = _new(stream, shape, dense, out_dtype or xt, x.device)
        made.append(out)
        ys = strides
    else:
        if out_dtype is not None and out.dtype is not out_dtype:
            raise ValueError("out must be of out_dtype")
        ys = _rows(out, shape, "out")
    yt = out.dtype
    rp = sp = None
    rs = ss = (0, 0)
    if residual is not None:
        if residual.dtype is not xt or sum_out is not None and sum_out.dtype is not xt:
            raise ValueError("residual and sum_out must be like x")
        rs, rp = _rows(residual, shape, "residual"), residual.data_ptr()
        if sum_out is None:
            sum_out = _new(stream, shape, dense, xt, x.device)
            made.append(sum_out)
            ss = strides
        else:
            ss = _rows(sum_out, shape, "sum_out")
        sp = sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    scales = qp = None
    if yt in _EIGHT:
        g = group or d
        if g < 1 or d % g:
            raise ValueError("group must divide the features")
        n = d // g
        scales = _new(stream, (*shape[:-1], n), (n, 1) if len(shape) == 2 else (H * n, n, 1), torch.float32,
                      x.device)
        made.append(scales)
        qp = scales.data_ptr()
    if H == 0:
        T, H = 0, 1
    _check(_library().rms_norm(x.data_ptr(), dt, T, H, d, *xs, rp, *rs, sp, *ss, wp or None, wt, unit_offset,
                               eps, out.data_ptr(), _DTYPE.get(yt, 0), *ys, qp, group, _stream(stream, x)))
    if stream is not None:
        _used(stream, made, [t for t in (out, sum_out) if not any(t is m for m in made)])
    if scales is None:
        return out if residual is None else (out, sum_out)
    return (out, scales) if residual is None else (out, scales, sum_out)


def linear4(x: torch.Tensor, codes: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor,
            x_scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, O] = x [T, K] times 4-bit weights in the checkpoint's layout: codes uint8
    [O, K / 2] (the even k in the low nibble), scale and bias fp16 or bf16 [O, K / group],
    group a multiple of 64.

    x is bf16 or fp16 (y of its type unless ``out_dtype`` says otherwise), or e4m3 or int8
    with ``x_scale`` fp32 [T, K / x_group] (y is bf16 unless told), as rms_norm returns
    them.  Made for a decode batch: every 16 tokens (8 where K is above 16384) read the weights
    anew, and beyond 16 to 32 tokens a matrix product of 16-bit weights is the faster one."""
    if x.dim() != 2 or codes.dim() != 2 or scale.dim() != 2:
        raise ValueError("x, codes and scale must have two axes")
    T, K = x.shape
    O = codes.shape[0]
    if codes.dtype is not torch.uint8 or codes.shape[1] * 2 != K or not codes.is_contiguous():
        raise ValueError("codes must be dense uint8 [O, K / 2]")
    if (scale.shape[0] != O or bias.shape != scale.shape or bias.dtype is not scale.dtype
            or scale.dtype not in _SCALE or not scale.is_contiguous() or not bias.is_contiguous()):
        raise ValueError("scale and bias must be dense [O, K / group] of fp16 or of bf16")
    ng = scale.shape[1]
    if ng < 1 or K % ng:
        raise ValueError("scale must have one column a group of K")
    _placed(x, codes, scale, bias, x_scale, out)
    if K > 1 and x.stride(1) != 1:
        raise ValueError("x's features must be contiguous")
    xg = 0
    if x.dtype in _EIGHT:
        if (x_scale is None or x_scale.dtype is not torch.float32 or x_scale.dim() != 2
                or x_scale.shape[0] != T or not x_scale.is_contiguous() or x_scale.shape[1] < 1
                or K % x_scale.shape[1]):
            raise ValueError("x_scale must be dense fp32 [T, K / group] for an 8-bit x")
        xg = K // x_scale.shape[1]
    elif x_scale is not None:
        raise ValueError("x_scale belongs to an 8-bit x")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16 if xg else x.dtype
    made = out is None
    if made:
        out = _new(stream, (T, O), (max(O, 1), 1), out_dtype, x.device)
    elif out.shape != (T, O) or out.dtype is not out_dtype or (O > 1 and out.stride(1) != 1):
        raise ValueError("out must be [T, O] of out_dtype, rows contiguous")
    if O == 0:
        return out
    # (the stride of a single row is never stepped along)
    _check(_library().linear4(
        x.data_ptr(), _DTYPE.get(x.dtype, 0), T, K, x.stride(0) if T > 1 else 0,
        None if x_scale is None else x_scale.data_ptr(), xg, codes.data_ptr(), scale.data_ptr(),
        bias.data_ptr(), _SCALE[scale.dtype], O, K // ng, out.data_ptr(), _DTYPE.get(out_dtype, 0),
        out.stride(0), _stream(stream, x)))
    if stream is not None:
        _used(stream, [out] if made else (), () if made else [out])
    return out


def _setting(v, dtype, B, name):
    """A row's setting as the address of a tensor [B], or as one number for all."""
    if not isinstance(v, torch.Tensor):
        return None, v
    if v.dtype is not dtype or v.dim() != 1 or v.shape[0] != B or not v.is_contiguous():
        raise ValueError(f"{name} must be a number or dense {dtype} [B]")
    return v.data_ptr(), 0


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           return_logprobs: bool = False, out: torch.Tensor | None = None, stream=None):
    """The next token of every row of logits [B, V] (bf16, fp16 or fp32), int32 [B], drawn
    with the random numbers u fp32 [B] in [0, 1): temperature (0: the largest logit), then
    top-k (0: off), top-p and min-p; each a number or a tensor [B] (top_k int32, the others
    fp32).  include/step.h has the definition, ties and rows without a token (-1) included.
    ``return_logprobs``: also the logarithm of the probability each was drawn with."""
    if logits.dim() != 2:
        raise ValueError("logits must be [B, V]")
    B, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("a row's logits must be contiguous")
    if u.dtype is not torch.float32 or u.dim() != 1 or u.shape[0] != B or not u.is_contiguous():
        raise ValueError("u must be dense fp32 [B]")
    _placed(logits, u, out, *[v for v in (temperature, top_k, top_p, min_p) if isinstance(v, torch.Tensor)])
    t, t0 = _setting(temperature, _F32, B, "temperature")
    k, k0 = _setting(top_k, torch.int32, B, "top_k")
    p, p0 = _setting(top_p, _F32, B, "top_p")
    m, m0 = _setting(min_p, _F32, B, "min_p")
    made = []
    if out is None:
        out = _new(stream, (B,), (1,), torch.int32, logits.device)
        made.append(out)
    else:
        _i32(out, 1, "out")
        _need(out.shape[0] == B and out.is_contiguous(), "out must be dense [B]")
    lp = None
    if return_logprobs:
        lp = _new(stream, (B,), (1,), _F32, logits.device)
        made.append(lp)
    _check(_library().sample(logits.data_ptr(), _DTYPE.get(logits.dtype, 0), B, V, logits.stride(0),
                             u.data_ptr(), t, k, p, m, t0, max(min(k0, 0x7fffffff), -1), p0, m0,
                             out.data_ptr(), None if lp is None else lp.data_ptr(),
                             _stream(stream, logits)))
    if stream is not None:
        _used(stream, made, () if made and made[0] is out else [out])
    return (out, lp) if return_logprobs else out
