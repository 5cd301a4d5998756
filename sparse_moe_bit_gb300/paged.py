"""Binding of include/paged.h: rotary positions, the paged key/value cache and
attention over it (argument marshalling only; no fallback path).

Tensors are CUDA tensors; shapes, types and strides are checked here, values
that only the GPU can see are handled by the kernels (include/paged.h says
how).  Every call enqueues on ``stream`` (default: torch's current one)."""
from __future__ import annotations

import ctypes

import torch

from . import moe as _moe

PAGED_DEVERR_WAIT_TIMEOUT = 1
PAGED_DEVERR_PAGE = 2

# names of the functions include/paged.h declares (checked by its ABI test)
EXPORTS = ["rope", "rope_frequencies", "rope_append", "paged_attention_workspace",
           "paged_attention", "pages_fork", "pages_reserve", "pages_free", "pages_compact",
           "pages_copy", "paged_get_device_error"]

_DTYPE = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}
SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("pages", ctypes.c_int), ("page", ctypes.c_int), ("heads", ctypes.c_int),
                ("dim", ctypes.c_int), ("page_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Batch(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("N", ctypes.c_int), ("T", ctypes.c_int),
                ("width", ctypes.c_int), ("table_stride", ctypes.c_int64)]


_lib = None


def _library():
    global _lib
    if _lib is not None:
        return _lib
    lib = _moe.load_library()
    P, I, L, F, D = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                     ctypes.c_double)
    C, B = ctypes.POINTER(_Cache), ctypes.POINTER(_Batch)
    sig = {
        "rope": [P, P, I, I, I, I, L, L, L, L, P, P, I, F, I, I, P],
        "rope_frequencies": [I, D, I, D, D, D, D, P, P],
        "rope_append": [P, L, P, I, P, L, P, L, C, B, P, I, F, I, P],
        "paged_attention_workspace": [C, B, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)],
        "paged_attention": [P, L, L, I, C, B, F, I, I, I, I, P, L, L, P, P, ctypes.c_size_t, P],
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
    _need(t.dtype is torch.int32 and t.dim() == ndim, f"{name} must be int32 with {ndim} axes")
    _need(t.shape[-1] <= 1 or t.stride(-1) == 1, f"{name} must be contiguous along its last axis")


def _cache(k, v):
    _need(k.dim() == 4 and k.dtype is v.dtype and k.shape == v.shape and k.stride() == v.stride(),
          "k_pages and v_pages must be [pages, page, heads, dim] of one type, shape and strides")
    _need(k.stride(3) == 1, "a head's features must be contiguous")
    s = k.stride()
    return _Cache(k.data_ptr(), v.data_ptr(), _DTYPE.get(k.dtype, 0), k.shape[0], k.shape[1],
                  k.shape[2], k.shape[3], s[0], s[1], s[2])


def _batch(table, cu_q, kv_len, T):
    _i32(table, 2, "table")
    _i32(cu_q, 1, "cu_q")
    _i32(kv_len, 1, "kv_len")
    n = table.shape[0]
    _need(cu_q.shape[0] == n + 1 and kv_len.shape[0] == n, "cu_q is [N + 1], kv_len [N], table [N, width]")
    return _Batch(table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), n, T, table.shape[1],
                  table.stride(0))


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original: int = 0, low: float = 1.0,
                     high: float = 32.0, device=None):
    """Radians a position of every pair (fp64 [rotary_dim / 2] on ``device``) and
    the factor on cos and sin: plain, or scaled ("linear", "ntk", "yarn",
    "banded"; include/paged.h has the formulas) for contexts ``factor`` times
    the ``original`` length."""
    _need(scaling in SCALINGS, f"unknown scaling {scaling!r}")
    f = torch.empty(max(rotary_dim // 2, 1), dtype=torch.float64)
    m = ctypes.c_double(1.0)
    _moe._check(_library().rope_frequencies(rotary_dim, base, SCALINGS[scaling], factor,
                                            float(original), low, high, f.data_ptr(),
                                            ctypes.byref(m)))
    return (f if device is None else f.to(device)), m.value


def rope(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, mscale: float = 1.0,
         interleaved: bool = False, inverse: bool = False, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Turn the first ``2 * len(freq)`` features of every head of x [T, H, D]
    (bf16, fp16 or fp32) by its token's position.  ``inverse`` turns back: the
    gradient of the call.  ``out`` may be x."""
    _need(x.dim() == 3 and x.dtype in _DTYPE, "x must be [T, H, D] of bf16, fp16 or fp32")
    T, H, D = x.shape
    _i32(positions, 1, "positions")
    _need(positions.shape[0] == T, "one position a token")
    _need(freq.dtype is torch.float64 and freq.dim() == 1 and freq.is_contiguous(), "freq must be fp64 [r]")
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    _need(out.shape == x.shape and out.dtype is x.dtype, "out must be like x")
    _need(D == 1 or (x.stride(2) == 1 and out.stride(2) == 1), "features must be contiguous")
    _moe._check(_library().rope(x.data_ptr(), out.data_ptr(), _DTYPE[x.dtype], T, H, D,
                                x.stride(0), x.stride(1), out.stride(0), out.stride(1),
                                positions.data_ptr(), freq.data_ptr(), freq.shape[0], mscale,
                                interleaved, inverse, _moe._stream(stream)))
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
    c = _cache(k_pages, v_pages)
    for t, h in ((q, Hq), (k, c.heads), (v, c.heads)):
        _need(t.dtype is k_pages.dtype and t.shape == (T, h, c.dim), "q, k, v must match the cache's type, heads and dim")
        _need(t.stride(2) == 1 and (h == 1 or t.stride(1) == D), "heads must be D apart")
    _need(freq.dtype is torch.float64 and freq.dim() == 1 and freq.is_contiguous(), "freq must be fp64 [r]")
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
    _need(q_out.shape == q.shape and q_out.dtype is q.dtype and q_out.is_contiguous(), "q_out must be dense and like q")
    b = _batch(table, cu_q, kv_len, T)
    _moe._check(_library().rope_append(
        q.data_ptr(), q.stride(0), q_out.data_ptr(), Hq, k.data_ptr(), k.stride(0), v.data_ptr(),
        v.stride(0), ctypes.byref(c), ctypes.byref(b), freq.data_ptr(), freq.shape[0], mscale,
        interleaved, _moe._stream(stream)))
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
    T, Hq, D = q.shape
    c = _cache(k_pages, v_pages)
    _need(q.dtype is k_pages.dtype and D == c.dim, "q must match the cache's type and dim")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
    _need(out.shape == q.shape and out.dtype is q.dtype, "out must be like q")
    _need(q.stride(2) == 1 and out.stride(2) == 1, "features must be contiguous")
    b = _batch(table, cu_q, kv_len, T)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    if scale is None:
        scale = D ** -0.5
    need = ctypes.c_size_t(0)
    _moe._check(lib.paged_attention_workspace(ctypes.byref(c), ctypes.byref(b), Hq, window, max_q,
                                              max_kv, ctypes.byref(need)))
    if workspace is None and need.value:
        workspace = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _moe._check(lib.paged_attention(
        q.data_ptr(), q.stride(0), q.stride(1), Hq, ctypes.byref(c), ctypes.byref(b), scale, causal,
        window, max_q, max_kv, out.data_ptr(), out.stride(0), out.stride(1),
        None if lse is None else lse.data_ptr(),
        None if workspace is None else workspace.data_ptr(), size, _moe._stream(stream)))
    return (out, lse) if return_lse else out


def _state(refs, table, lens=None):
    _i32(refs, 1, "refs")
    _i32(table, 2, "table")
    if lens is not None:
        _i32(lens, 1, "lens")
        _need(lens.shape[0] == table.shape[0], "one length a slot of the table")
    return refs.data_ptr(), refs.shape[0], table.data_ptr(), table.stride(0), table.shape[1]


def pages_fork(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, src: torch.Tensor,
               dst: torch.Tensor, refused: torch.Tensor | None = None, stream=None) -> None:
    """Slot dst[i] of the table becomes a copy of slot src[i] that shares its
    pages (refs int32 [P], table int32 [S, width], lens int32 [S], in place).
    ``refused``: int32 [1], the number of pairs left out."""
    st = _state(refs, table, lens)
    _i32(src, 1, "src")
    _i32(dst, 1, "dst")
    _need(src.shape == dst.shape, "src and dst must have one length")
    _moe._check(_library().pages_fork(*st, lens.data_ptr(), lens.shape[0], src.data_ptr(),
                                      dst.data_ptr(), src.shape[0],
                                      None if refused is None else refused.data_ptr(),
                                      _moe._stream(stream)))


def pages_reserve(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, add: torch.Tensor,
                  page: int, stream=None):
    """Room for add[s] more tokens in every slot, in place; a slot whose partly
    filled last page is shared gets one of its own.  Returns moves int32 [S, 2]
    (the page to copy from and to, or -1, -1: hand them to pages_copy) and
    status int32 [2] (pages missing, slots whose row is too short; nothing was
    changed unless both are 0)."""
    st = _state(refs, table, lens)
    _i32(add, 1, "add")
    S = lens.shape[0]
    _need(add.shape[0] == S, "one number a slot")
    buf = torch.empty(3 * S + 3, dtype=torch.int32, device=refs.device)
    moves, status, scratch = buf[:2 * S].view(S, 2), buf[2 * S:2 * S + 2], buf[2 * S + 2:]
    _moe._check(_library().pages_reserve(*st, lens.data_ptr(), add.data_ptr(), S, page,
                                         moves.data_ptr(), status.data_ptr(), scratch.data_ptr(),
                                         _moe._stream(stream)))
    return moves, status


def pages_free(refs: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, slots: torch.Tensor,
               stream=None) -> None:
    """The slots give up their pages, in place."""
    st = _state(refs, table, lens)
    _i32(slots, 1, "slots")
    _moe._check(_library().pages_free(*st, lens.data_ptr(), lens.shape[0], slots.data_ptr(),
                                      slots.shape[0], _moe._stream(stream)))


def pages_compact(refs: torch.Tensor, table: torch.Tensor, stream=None):
    """Renumber the pages in use to the lowest numbers, in place.  Returns moves
    int32 [P, 2] and their count (int32 scalar), for pages_copy."""
    st = _state(refs, table)
    P = refs.shape[0]
    buf = torch.empty(3 * P + 2, dtype=torch.int32, device=refs.device)
    moves, count, scratch = buf[:2 * P].view(P, 2), buf[2 * P], buf[2 * P + 1:]
    _moe._check(_library().pages_compact(*st, table.shape[0], moves.data_ptr(), count.data_ptr(),
                                         scratch.data_ptr(), _moe._stream(stream)))
    return moves, count


def pages_copy(pools: torch.Tensor, moves: torch.Tensor, count: torch.Tensor | None = None,
               stream=None) -> None:
    """Copy the rows of page moves[i, 0] to page moves[i, 1] in every array of
    pools [B, P, ...] (keys and values of all layers; what a page holds is
    contiguous).  ``count``: only the first so many moves (int32, on the GPU)."""
    _need(pools.dim() >= 3, "pools must be [B, P, ...]")
    _i32(moves, 2, "moves")
    _need(moves.shape[1] == 2 and (moves.shape[0] <= 1 or moves.stride(0) == 2), "moves must be dense [M, 2]")
    es = pools.element_size()
    n = 1
    for size, stride in zip(reversed(pools.shape[2:]), reversed(pools.stride()[2:])):
        _need(size == 1 or stride == n, "a page's rows must be contiguous")
        n *= size
    _need(count is None or count.dtype is torch.int32, "count must be int32")
    _moe._check(_library().pages_copy(pools.data_ptr(), pools.shape[0], pools.stride(0) * es,
                                      pools.shape[1], pools.stride(1) * es, n * es,
                                      moves.data_ptr(), moves.shape[0],
                                      None if count is None else count.data_ptr(),
                                      _moe._stream(stream)))


def paged_device_error(stream=None) -> int:
    """Read and clear the error word of these calls (PAGED_DEVERR_* bits);
    synchronises the stream."""
    code = ctypes.c_int(0)
    st = _library().paged_get_device_error(_moe._stream(stream), ctypes.byref(code))
    if st not in (0, 5):
        _moe._check(st)
    return code.value
