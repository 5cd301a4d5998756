"""Binding of include/step.h: the residual's addition with the RMS norm, products
with 4-bit weights, and the choice of the next token (argument marshalling only;
no fallback path).

Tensors are CUDA tensors of the current device; that, shapes, types and strides
are checked here.  Every call enqueues on ``stream`` (default: torch's current
one); on a given stream outputs come from that stream's pool.  Like the package's
other calls they leave no autograd graph."""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import moe as _moe
from .paged import _check, _i32, _need, _new, _placed, _stream, _torch_stream, _used

# names of the functions include/step.h declares (checked by its ABI test)
EXPORTS = ["rms_norm", "linear4", "sample"]

_DTYPE = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3, torch.float8_e4m3fn: 4,
          torch.int8: 5}
_EIGHT = (torch.float8_e4m3fn, torch.int8)
_SCALE = {torch.float16: _moe.MOE_SCALE_F16, torch.bfloat16: _moe.MOE_SCALE_BF16}
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
        "sample": [P, I, I, I, L, P, P, P, P, P, P, P, P],
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
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{name}'s features must be contiguous")
    return (st[0], st[1]) if len(shape) == 3 else (st[0], 0)


def _dense(shape):
    st, n = [], 1
    for x in reversed(shape):
        st.append(n)
        n *= max(x, 1)
    return tuple(reversed(st))


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
             residual: torch.Tensor | None = None, eps: float = 1e-6, unit_offset: bool = False,
             out_dtype: torch.dtype | None = None, group: int = 0,
             out: torch.Tensor | None = None, sum_out: torch.Tensor | None = None, stream=None):
    """RMS norm over the last axis of x [T, d] or [T, H, d] (bf16, fp16 or fp32; any
    strides over the first axes), after the addition of ``residual``; all in fp32.

    ``weight`` [d] of x's type or fp32 (``unit_offset``: 1 + weight).  Returns
    y of ``out_dtype`` (default x's); of torch.float8_e4m3fn or torch.int8: y and its
    scales, fp32 [..., d / group], one for ``group`` features (0: a row); and behind
    them, with a residual, x + residual in x's type.  ``out`` may be x, ``sum_out``
    x or the residual (in place)."""
    shape = x.shape
    dt = _DTYPE.get(x.dtype, 0)
    if dt not in (1, 2, 3) or len(shape) not in (2, 3):
        raise ValueError("x must be [T, d] or [T, H, d] of bf16, fp16 or fp32")
    T, H, d = shape[0], shape[1] if len(shape) == 3 else 1, shape[-1]
    _placed(x, weight, residual, out, sum_out)
    xs = _rows(x, shape, "x")
    if weight is not None and (weight.dim() != 1 or weight.shape[0] != d or not weight.is_contiguous()):
        raise ValueError("weight must be dense [d]")
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    yt = _DTYPE.get(out_dtype, 0)
    if out is not None and out.dtype is not out_dtype:
        raise ValueError("out must be of out_dtype")
    made = []
    if out is None:
        out = _new(stream, shape, _dense(shape), out_dtype, x.device)
        made.append(out)
    ys = _rows(out, shape, "out")
    rs = ss = (0, 0)
    if residual is not None:
        if residual.dtype is not x.dtype:
            raise ValueError("residual must be like x")
        rs = _rows(residual, shape, "residual")
        if sum_out is None:
            sum_out = _new(stream, shape, _dense(shape), x.dtype, x.device)
            made.append(sum_out)
        elif sum_out.dtype is not x.dtype:
            raise ValueError("sum_out must be like x")
        ss = _rows(sum_out, shape, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out without a residual")
    scales = None
    if out_dtype in _EIGHT:
        g = group or d
        if g < 1 or d % g:
            raise ValueError("group must divide the features")
        s_shape = (*shape[:-1], d // g)
        scales = _new(stream, s_shape, _dense(s_shape), torch.float32, x.device)
        made.append(scales)
    if H == 0:
        T, H = 0, 1
    _check(_library().rms_norm(
        x.data_ptr(), dt, T, H, d, *xs, None if residual is None else residual.data_ptr(), *rs,
        None if sum_out is None else sum_out.data_ptr(), *ss,
        None if weight is None else weight.data_ptr(),
        0 if weight is None else _DTYPE.get(weight.dtype, 0), unit_offset, eps, out.data_ptr(), yt,
        *ys, None if scales is None else scales.data_ptr(), group, _stream(stream, x)))
    if stream is not None:
        _used(stream, made, [t for t in (out, sum_out) if not any(t is m for m in made)])
    res = (out,) if scales is None else (out, scales)
    if residual is not None:
        res += (sum_out,)
    return res if len(res) > 1 else out


def linear4(x: torch.Tensor, codes: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor,
            x_scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, O] = x [T, K] times 4-bit weights in the checkpoint's layout: codes uint8
    [O, K / 2] (the even k in the low nibble), scale and bias fp16 or bf16 [O, K / group],
    group a multiple of 64.

    x is bf16 or fp16 (y of its type unless ``out_dtype`` says otherwise), or e4m3 or int8
    with ``x_scale`` fp32 [T, K / x_group] (y is bf16 unless told), as rms_norm returns
    them.  Made for a decode batch: the weights are read once for every 64 tokens."""
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


def _setting(v, off, dtype, B, name, like):
    """A row's setting: None where it is off for all, else a tensor [B]."""
    if v is None or (not isinstance(v, torch.Tensor) and v == off):
        return None
    if not isinstance(v, torch.Tensor):
        return torch.full((B,), v, dtype=dtype, device=like.device)
    if v.dtype is not dtype or v.dim() != 1 or v.shape[0] != B or not v.is_contiguous():
        raise ValueError(f"{name} must be a number or dense {dtype} [B]")
    return v


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
    f32, tens = torch.float32, [t for t in (temperature, top_k, top_p, min_p) if isinstance(t, torch.Tensor)]
    _placed(logits, u, out, *tens)
    # (numbers become tensors of the stream that reads them)
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(_torch_stream(stream)):
        t = _setting(temperature, 1.0, f32, B, "temperature", logits)
        k = _setting(top_k, 0, torch.int32, B, "top_k", logits)
        p = _setting(top_p, 1.0, f32, B, "top_p", logits)
        m = _setting(min_p, 0.0, f32, B, "min_p", logits)
    made = []
    if out is None:
        out = _new(stream, (B,), (1,), torch.int32, logits.device)
        made.append(out)
    else:
        _i32(out, 1, "out")
        _need(out.shape[0] == B and out.is_contiguous(), "out must be dense [B]")
    lp = None
    if return_logprobs:
        lp = _new(stream, (B,), (1,), f32, logits.device)
        made.append(lp)
    ptr = lambda x: None if x is None else x.data_ptr()
    _check(_library().sample(logits.data_ptr(), _DTYPE.get(logits.dtype, 0), B, V, logits.stride(0),
                             u.data_ptr(), ptr(t), ptr(k), ptr(p), ptr(m), out.data_ptr(), ptr(lp),
                             _stream(stream, logits)))
    if stream is not None:
        _used(stream, made, () if made and made[0] is out else [out])
    return (out, lp) if return_logprobs else out
