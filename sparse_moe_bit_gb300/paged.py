"""Binding of include/paged.h: rotary positions, the paged key/value cache and
attention over it (argument marshalling only; no fallback path).

Tensors are CUDA tensors of the current device; that, shapes, types and strides
are checked here, values that only the GPU can see are handled by the kernels
(include/paged.h says how).  Every call enqueues on ``stream`` (default: torch's
current one).  Like the package's other calls they leave no autograd graph: a
gradient is a call of its own (rope's is rope with ``inverse``)."""
from __future__ import annotations

import ctypes
import struct

import torch

from . import moe as _moe

PAGED_DEVERR_WAIT_TIMEOUT = 1
PAGED_DEVERR_PAGE = 2
PAGED_DEVERR_LENGTH = 4

# names of the functions include/paged.h declares (checked by its ABI test)
EXPORTS = ["rope", "rope_frequencies", "rope_append", "paged_attention_workspace",
           "paged_attention", "paged_attention_shared_workspace", "paged_attention_shared", "pages_fork", "pages_reserve", "pages_free", "pages_compact",
           "pages_copy", "paged_get_device_error"]

_DTYPE = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}
SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}


# paged_cache and paged_batch of include/paged.h, packed (the calls of a decode
# step are over in a few microseconds: building ctypes structures would double
# their host time)
_CACHE = struct.Struct("@PPiiiiiqqq")
_BATCH = struct.Struct("@PPPiiiq")


_lib = None
_sizes: dict = {}  # workspace bytes of paged_attention by the call's sizes


def _check(status):
    if status:
        _moe._check(status)



def _library():
    global _lib
    if _lib is not None:
        return _lib
    lib = _moe.load_library()
    P, I, L, F, D = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                     ctypes.c_double)
    C = B = ctypes.c_char_p
    sig = {
        "rope": [P, P, I, I, I, I, L, L, L, L, P, P, I, F, I, I, P],
        "rope_frequencies": [I, D, I, D, D, D, D, P, P],
        "rope_append": [P, L, P, I, P, L, P, L, C, B, P, I, F, I, P],
        "paged_attention_workspace": [C, B, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)],
        "paged_attention": [P, L, L, I, C, B, F, I, I, I, I, P, L, L, P, P, ctypes.c_size_t, P],
        "paged_attention_shared_workspace": [C, B, I, I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)],
        "paged_attention_shared": [P, L, L, I, C, B, P, P, I, F, I, I, I, I, I, P, L, L, P, P,
                                   ctypes.c_size_t, P],
        "pages_fork": [P, I, P, L, I, P, I, P, P, I, P, P],
        "pages_reserve": [P, I, P, L, I, P, P, I, I, P, P, P, P],
        "pages_free": [P, I, P, L, I, P, I, P, I, P],
        "pages_compact": [P, I, P, L, I, I, P, P, P, P],
        "pages_copy": [P, I, L, I, L, L, P, I, P, P],
        "paged_get_device_error": [P, ctypes.POINTER(I)],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    _lib = lib
    return lib


def _need(ok, msg):
    if not ok:
        raise ValueError(msg)


def _i32(t, ndim, name):
    if t.dtype is not torch.int32 or t.dim() != ndim:
        raise ValueError(f"{name} must be int32 with {ndim} axes")
    if not t.is_contiguous() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")


def _placed(t, *others):
    """Every tensor has to lie on the current device: the kernels run there, and an
    address of the host or of another device would be a memory fault in them.
    (Where there is no device at all the library says so.)"""
    d = t.get_device()
    if d != _current_device() if d >= 0 else _have_gpu():
        raise ValueError(f"tensors must be on the current GPU, not on {t.device}")
    for o in others:
        if o is not None and o.get_device() != d:
            raise ValueError(f"tensors must be on one GPU, not on {t.device} and {o.device}")


def _one(t, name):
    if t is not None and (t.dtype is not torch.int32 or t.numel() != 1):
        raise ValueError(f"{name} must be one int32")


def _stream(stream, t) -> int:
    """The raw stream: the given one, or torch's current one of t's device."""
    if stream is not None:
        return stream.cuda_stream
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    return _raw_stream(t.get_device())


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device
_have_gpu = torch.cuda.is_available


def _new(stream, shape, strides, dtype, device):
    """A tensor for the kernels on ``stream`` (None: the current one) to write.
    It comes from that stream's pool: a block of another stream's may still be in
    use there by work that was queued before its last holder let go of it."""
    if stream is None or device.type != "cuda":
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream)):
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _torch_stream(stream):
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream)


def _used(stream, made, given):
    """After a call on a given stream: what was made here goes back to the caller,
    whose current stream may read it last; what was given belongs to another stream
    and is used on this one.  The allocator is told of both."""
    if stream is None:
        return
    for t in made:
        if t is not None:
            t.record_stream(torch.cuda.current_stream(t.device))
    for t in given:
        if t is not None:
            t.record_stream(_torch_stream(stream))


def _cache(k, v):
    shape, st = k.shape, k.stride()
    if len(shape) != 4 or v.shape != shape or v.stride() != st or k.dtype is not v.dtype or st[3] != 1:
        raise ValueError("k_pages and v_pages must be [pages, page, heads, dim] of one type, shape "
                         "and strides, a head's features contiguous")
    return _CACHE.pack(k.data_ptr(), v.data_ptr(), _DTYPE.get(k.dtype, 0), *shape, *st[:3])


def _batch(table, cu_q, kv_len, T):
    _i32(table, 2, "table")
    _i32(cu_q, 1, "cu_q")
    _i32(kv_len, 1, "kv_len")
    n, width = table.shape
    if cu_q.shape[0] != n + 1 or kv_len.shape[0] != n:
        raise ValueError("cu_q is [N + 1], kv_len [N], table [N, width]")
    return _BATCH.pack(table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), n, T, width,
                       table.stride(0))


def _freq(freq):
    if freq.dtype is not torch.float64 or freq.dim() != 1 or not freq.is_contiguous():
        raise ValueError("freq must be fp64 [r]")
    return freq.data_ptr(), freq.shape[0]


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original: int = 0, low: float = 1.0,
                     high: float = 32.0, device=None):
    """Radians a position of every pair (fp64 [rotary_dim / 2] on ``device``, by
    default the host; rope and rope_append take them on the GPU) and the factor
    on cos and sin: plain, or scaled ("linear", "ntk", "yarn", "banded";
    include/paged.h has the formulas) for contexts ``factor`` times the
    ``original`` length."""
    _need(scaling in SCALINGS, f"unknown scaling {scaling!r}")
    f = torch.empty(max(rotary_dim // 2, 1), dtype=torch.float64)
    m = ctypes.c_double(1.0)
    _check(_library().rope_frequencies(rotary_dim, base, SCALINGS[scaling], factor,
                                            float(original), low, high, f.data_ptr(),
                                            ctypes.byref(m)))
    return (f if device is None else f.to(device)), m.value


def rope(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, mscale: float = 1.0,
         interleaved: bool = False, inverse: bool = False, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Turn the first ``2 * len(freq)`` features of every head of x [T, H, D]
    (bf16, fp16 or fp32) by its token's position.  ``inverse`` turns back: the
    gradient of the call.  ``out`` may be x."""
    dt = _DTYPE.get(x.dtype)
    if dt is None or x.dim() != 3:
        raise ValueError("x must be [T, H, D] of bf16, fp16 or fp32")
    T, H, D = x.shape
    _placed(x, positions, freq, out)
    _i32(positions, 1, "positions")
    if positions.shape[0] != T:
        raise ValueError("one position a token")
    f, r = _freq(freq)
    made = out is None
    if made:
        out = _new(stream, (T, H, D), (H * D, D, 1), x.dtype, x.device)
    elif out.shape != x.shape or out.dtype is not x.dtype:
        raise ValueError("out must be like x")
    xs, os_ = x.stride(), out.stride()
    if D > 1 and (xs[2] != 1 or os_[2] != 1):
        raise ValueError("features must be contiguous")
    _check(_library().rope(x.data_ptr(), out.data_ptr(), dt, T, H, D, xs[0], xs[1], os_[0], os_[1],
                           positions.data_ptr(), f, r, mscale, interleaved, inverse,
                           _stream(stream, x)))
    if stream is not None:
        _used(stream, [out] if made else (), () if made else [out])
    return out


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor,
                v_pages: torch.Tensor, table: torch.Tensor, cu_q: torch.Tensor,
                kv_len: torch.Tensor, freq: torch.Tensor, mscale: float = 1.0,
                interleaved: bool = False, q_out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Turn the new tokens' queries and keys by their positions in their
    sequences and write keys and values into the cache; returns the queries.

    q [T, Hq, D], k, v [T, Hk, D] (heads D apart; views of one projection's
    output will do), k_pages, v_pages [pages, page, Hk, D] (any strides over
    the first three axes, the same for both), table int32 [N, width], cu_q
    int32 [N + 1], kv_len int32 [N] (new tokens included), freq fp64 [r]."""
    T, Hq, D = q.shape
    _placed(q, k, v, k_pages, v_pages, table, cu_q, kv_len, freq, q_out)
    c = _cache(k_pages, v_pages)
    dt, hk = k_pages.dtype, k_pages.shape[2]
    kv = (T, hk, k_pages.shape[3])
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    if (D != kv[2] or k.shape != kv or v.shape != kv or q.dtype is not dt or k.dtype is not dt
            or v.dtype is not dt):
        raise ValueError("q, k, v must match the cache's type, heads and dim")
    if (qs[2] != 1 or ks[2] != 1 or vs[2] != 1 or (Hq > 1 and qs[1] != D)
            or (hk > 1 and (ks[1] != D or vs[1] != D))):
        raise ValueError("heads must be D apart")
    f, r = _freq(freq)
    made = q_out is None
    if made:
        q_out = _new(stream, (T, Hq, D), (Hq * D, D, 1), dt, q.device)
    elif q_out.shape != q.shape or q_out.dtype is not dt or not q_out.is_contiguous():
        raise ValueError("q_out must be dense and like q")
    _check(_library().rope_append(q.data_ptr(), qs[0], q_out.data_ptr(), Hq, k.data_ptr(), ks[0],
                                  v.data_ptr(), vs[0], c, _batch(table, cu_q, kv_len, T), f, r,
                                  mscale, interleaved, _stream(stream, q)))
    if stream is not None:
        _used(stream, [q_out] if made else (), () if made else [q_out])
    return q_out


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                    table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor,
                    scale: float | None = None, causal: bool = True, window: int = 0,
                    max_q: int = 0, max_kv: int = 0, return_lse: bool = False,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None):
    """Attention of the new tokens q [T, Hq, D] over the paged cache (arguments
    as for rope_append).  ``window`` > 0 keeps the last so many keys.  ``max_q``
    and ``max_kv`` (the longest chunk and context, if the caller knows them)
    choose the kernel and the split over the keys and bound nothing.  Returns
    out [T, Hq, D] and, with ``return_lse``, the fp32 logarithms of the
    softmax's sums [T, Hq].  ``workspace``: a byte tensor to use instead of one
    made here (paged_attention_workspace() in include/paged.h)."""
    lib = _library()
    if max(window, max_q, max_kv) > 0x7fffffff:  # beyond any context, and beyond an int
        window, max_q, max_kv = (min(x, 0x7fffffff) for x in (window, max_q, max_kv))
    T, Hq, D = q.shape
    _placed(q, k_pages, v_pages, table, cu_q, kv_len, out, workspace)
    c = _cache(k_pages, v_pages)
    if q.dtype is not k_pages.dtype or D != k_pages.shape[3]:
        raise ValueError("q must match the cache's type and dim")
    given = (out, workspace)
    if out is None:
        out = _new(stream, (T, Hq, D), (Hq * D, D, 1), q.dtype, q.device)
    elif out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError("out must be like q")
    qs, os_ = q.stride(), out.stride()
    if qs[2] != 1 or os_[2] != 1:
        raise ValueError("features must be contiguous")
    b = _batch(table, cu_q, kv_len, T)
    lse = _new(stream, (T, Hq), (Hq, 1), torch.float32, q.device) if return_lse else None
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        # (a function of these sizes alone, on one kind of GPU)
        key = (T, Hq, k_pages.dtype, *k_pages.shape[1:], *table.shape, window, max_q, max_kv)
        size, ws = _sizes.get(key), None
        if size is None:
            need = ctypes.c_size_t(0)
            _check(lib.paged_attention_workspace(c, b, Hq, window, max_q, max_kv, ctypes.byref(need)))
            if len(_sizes) >= 4096:
                _sizes.clear()
            size = _sizes[key] = need.value
        if size:
            workspace = _new(stream, (size,), (1,), torch.uint8, q.device)
            ws = workspace.data_ptr()
    else:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        size, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    _check(lib.paged_attention(q.data_ptr(), qs[0], qs[1], Hq, c, b, scale, causal, window, max_q,
                               max_kv, out.data_ptr(), os_[0], os_[1],
                               None if lse is None else lse.data_ptr(), ws, size,
                               _stream(stream, q)))
    if stream is not None:  # (a workspace made here is let go of on the stream that uses it)
        _used(stream, (lse,) if given[0] is out else (out, lse), given)
    return (out, lse) if return_lse else out


def paged_attention_shared(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                           table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor,
                           cu_group: torch.Tensor, shared: torch.Tensor,
                           scale: float | None = None, causal: bool = True, max_q: int = 0,
                           max_group: int = 0, max_shared: int = 0, max_tail: int = 0,
                           return_lse: bool = False, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None):
    """paged_attention for groups of adjacent sequences that share their first keys, which
    are read once a group: group g holds the sequences cu_group[g] .. cu_group[g + 1] - 1
    (int32 [groups + 1]), whose first shared[g] keys (int32 [groups]) are the same; they are
    read through the first one's row of the table.  ``max_q``, ``max_group``, ``max_shared``
    and ``max_tail`` (the longest chunk, the most new tokens of a group, the most keys of a
    group, the most keys of a sequence behind them, if the caller knows them) choose kernels
    and splits and bound nothing.  Faster than paged_attention once the shared keys and values,
    counted once for each sequence, are some 150 MB in groups of four and more; slower below,
    and where nothing is shared.  The rest is as for paged_attention;
    paged_attention_shared_workspace() in include/paged.h sizes ``workspace``."""
    lib = _library()
    if max(max_q, max_group, max_shared, max_tail) > 0x7fffffff:
        max_q, max_group, max_shared, max_tail = (min(x, 0x7fffffff) for x in
                                                  (max_q, max_group, max_shared, max_tail))
    T, Hq, D = q.shape
    _placed(q, k_pages, v_pages, table, cu_q, kv_len, cu_group, shared, out, workspace)
    c = _cache(k_pages, v_pages)
    if q.dtype is not k_pages.dtype or D != k_pages.shape[3]:
        raise ValueError("q must match the cache's type and dim")
    _i32(cu_group, 1, "cu_group")
    _i32(shared, 1, "shared")
    G = shared.shape[0]
    if cu_group.shape[0] != G + 1:
        raise ValueError("cu_group is [groups + 1], shared [groups]")
    given = (out, workspace)
    if out is None:
        out = _new(stream, (T, Hq, D), (Hq * D, D, 1), q.dtype, q.device)
    elif out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError("out must be like q")
    qs, os_ = q.stride(), out.stride()
    if qs[2] != 1 or os_[2] != 1:
        raise ValueError("features must be contiguous")
    b = _batch(table, cu_q, kv_len, T)
    lse = _new(stream, (T, Hq), (Hq, 1), torch.float32, q.device) if return_lse else None
    if scale is None:
        scale = D ** -0.5
    if workspace is None:
        key = (T, Hq, k_pages.dtype, *k_pages.shape[1:], *table.shape, G, max_q, max_group,
               max_shared, max_tail)
        size, ws = _sizes.get(key), None
        if size is None:
            need = ctypes.c_size_t(0)
            _check(lib.paged_attention_shared_workspace(c, b, Hq, G, max_q, max_group, max_shared,
                                                        max_tail, ctypes.byref(need)))
            if len(_sizes) >= 4096:
                _sizes.clear()
            size = _sizes[key] = need.value
        if size:
            workspace = _new(stream, (size,), (1,), torch.uint8, q.device)
            ws = workspace.data_ptr()
    else:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        size, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    _check(lib.paged_attention_shared(q.data_ptr(), qs[0], qs[1], Hq, c, b, cu_group.data_ptr(),
                                      shared.data_ptr(), G, scale, causal, max_q, max_group,
                                      max_shared, max_tail, out.data_ptr(), os_[0], os_[1],
                                      None if lse is None else lse.data_ptr(), ws, size,
                                      _stream(stream, q)))
    if stream is not None:
        _used(stream, (lse,) if given[0] is out else (out, lse), given)
    return (out, lse) if return_lse else out


def _state(refs, table, lens=None):
    _i32(refs, 1, "refs")
    _i32(table, 2, "table")
    if lens is not None:
        _i32(lens, 1, "lens")
        if lens.shape[0] != table.shape[0]:
            raise ValueError("one length a slot of the table")
    return refs.data_ptr(), refs.shape[0], table.data_ptr(), table.stride(0), table.shape[1]


def pages_fork(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, src: torch.Tensor,
               dst: torch.Tensor, refused: torch.Tensor | None = None, stream=None) -> None:
    """Slot dst[i] of the table becomes a copy of slot src[i] that shares its
    pages (refs int32 [P], table int32 [S, width], lens int32 [S], in place).
    ``refused``: int32 [1], the number of pairs left out."""
    _placed(refs, table, lens, src, dst, refused)
    st = _state(refs, table, lens)
    _i32(src, 1, "src")
    _i32(dst, 1, "dst")
    if src.shape != dst.shape:
        raise ValueError("src and dst must have one length")
    _one(refused, "refused")
    _check(_library().pages_fork(*st, lens.data_ptr(), lens.shape[0], src.data_ptr(),
                                      dst.data_ptr(), src.shape[0],
                                      None if refused is None else refused.data_ptr(),
                                      _stream(stream, refs)))


def pages_reserve(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, add: torch.Tensor,
                  page: int, stream=None):
    """Room for add[s] more tokens in every slot, in place; a slot whose partly
    filled last page is shared gets one of its own.  Returns moves int32 [S, 2]
    (the page to copy from and to, or -1, -1: hand them to pages_copy) and
    status int32 [2] (pages missing, slots whose row is too short; nothing was
    changed unless both are 0)."""
    _placed(refs, table, lens, add)
    st = _state(refs, table, lens)
    _i32(add, 1, "add")
    S = lens.shape[0]
    if add.shape[0] != S:
        raise ValueError("one number a slot")
    buf = _new(stream, (3 * S + 3,), (1,), torch.int32, refs.device)  # moves, status, scratch
    moves, status = buf.as_strided((S, 2), (2, 1)), buf.as_strided((2,), (1,), 2 * S)
    at = buf.data_ptr()
    _check(_library().pages_reserve(*st, lens.data_ptr(), add.data_ptr(), S, page,
                                         at, at + 8 * S, at + 8 * S + 8,
                                         _stream(stream, refs)))
    _used(stream, (buf,), ())
    return moves, status


def pages_free(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, slots: torch.Tensor,
               stream=None) -> None:
    """The slots give up their pages, in place."""
    _placed(refs, table, lens, slots)
    st = _state(refs, table, lens)
    _i32(slots, 1, "slots")
    _check(_library().pages_free(*st, lens.data_ptr(), lens.shape[0], slots.data_ptr(),
                                      slots.shape[0], _stream(stream, refs)))


def pages_compact(refs: torch.Tensor, table: torch.Tensor, stream=None):
    """Renumber the pages in use to the lowest numbers, in place.  Returns moves
    int32 [P, 2] and their count (int32 scalar), for pages_copy."""
    _placed(refs, table)
    st = _state(refs, table)
    P = refs.shape[0]
    buf = _new(stream, (3 * P + 2,), (1,), torch.int32, refs.device)  # moves, count, scratch
    moves, count = buf.as_strided((P, 2), (2, 1)), buf.as_strided((), (), 2 * P)
    at = buf.data_ptr()
    _check(_library().pages_compact(*st, table.shape[0], at, at + 8 * P,
                                         at + 8 * P + 4, _stream(stream, refs)))
    _used(stream, (buf,), ())
    return moves, count


def pages_copy(pools: torch.Tensor, moves: torch.Tensor, count: torch.Tensor | None = None,
               stream=None) -> None:
    """Copy the rows of page moves[i, 0] to page moves[i, 1] in every array of
    pools [B, P, ...] (keys and values of all layers; what a page holds is
    contiguous).  ``count``: only the first so many moves (int32, on the GPU)."""
    shape, st, es = pools.shape, pools.stride(), pools.element_size()
    if len(shape) < 3:
        raise ValueError("pools must be [B, P, ...]")
    _placed(pools, moves, count)
    _i32(moves, 2, "moves")
    if moves.shape[1] != 2 or (moves.shape[0] > 1 and moves.stride(0) != 2):
        raise ValueError("moves must be dense [M, 2]")
    n = 1
    for i in range(len(shape) - 1, 1, -1):
        if shape[i] != 1 and st[i] != n:
            raise ValueError("a page's rows must be contiguous")
        n *= shape[i]
    _one(count, "count")
    _check(_library().pages_copy(pools.data_ptr(), shape[0], st[0] * es, shape[1], st[1] * es,
                                 n * es, moves.data_ptr(), moves.shape[0],
                                 None if count is None else count.data_ptr(),
                                 _stream(stream, pools)))


def paged_device_error(stream=None) -> int:
    """Read and clear the error word of these calls (PAGED_DEVERR_* bits);
    synchronises the stream."""
    code = ctypes.c_int(0)
    st = _library().paged_get_device_error(_moe._stream(stream), ctypes.byref(code))
    if st not in (0, 5):
        _check(st)
    return code.value
