"""paged_attention_shared: refusals of bad arguments before anything could be enqueued.  No GPU."""
import ctypes
import math

import pytest

from tests.test_paged_abi import _A, BATCH_BAD, CACHE_BAD, _batch, _cache, lib  # noqa: F401


def _attend(lib, c=None, b=None, **kw):
    a = dict(q=_A, q_ts=1024, q_hs=128, Hq=8, cu_group=_A, shared=_A, groups=1, scale=0.1, causal=1, max_q=1,
             max_group=2, max_shared=32, max_tail=32, o=_A, o_ts=1024, o_hs=128, lse=None, ws=_A, ws_bytes=1 << 40)
    a.update(kw)
    v = list(a.values())
    return lib.paged_attention_shared(*v[:4], c or _cache(), b or _batch(), *v[4:], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(q=_A + 8), 1), (dict(q_ts=1020), 1), (dict(o_hs=-128), 1),
    (dict(Hq=0), 1), (dict(Hq=7), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1), (dict(max_q=-1), 1),
    (dict(max_group=-1), 1), (dict(max_shared=-1), 1), (dict(max_tail=-2), 1), (dict(groups=-1), 1),
    (dict(lse=_A + 2), 1), (dict(ws=_A + 8), 1), (dict(ws=None), 1), (dict(ws_bytes=0), 1), (dict(cu_group=None), 1),
    (dict(shared=None), 1), (dict(cu_group=_A + 2), 1), (dict(shared=_A + 1), 1)])
def test_bad_arguments(lib, kw, status):  # noqa: F811
    assert _attend(lib, **kw) == status, lib.moe_last_error()
    assert lib.moe_last_error()


@pytest.mark.parametrize("kw,status", CACHE_BAD)
def test_bad_cache(lib, kw, status):  # noqa: F811
    assert _attend(lib, c=_cache(**kw)) == status
    n = ctypes.c_size_t()
    assert lib.paged_attention_shared_workspace(_cache(**kw), _batch(), 8, 1, 0, 0, 0, 0, ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status", BATCH_BAD)
def test_bad_batch(lib, kw, status):  # noqa: F811
    assert _attend(lib, b=_batch(**kw)) == status


def test_workspace(lib):  # noqa: F811
    n, plain = ctypes.c_size_t(), ctypes.c_size_t()
    c, b = _cache(pages=4096), _batch(N=2, T=2, width=4096, table_stride=4096)
    for hints in ((0, 0, 0, 0), (1, 2, 60000, 100), (1, 2, 16, 60000)):
        assert lib.paged_attention_shared_workspace(c, b, 8, 1, *hints, ctypes.byref(n)) == 0
        kw = dict(zip(("max_q", "max_group", "max_shared", "max_tail"), hints))
        assert n.value > 0 and _attend(lib, c=c, b=b, ws_bytes=n.value - 1, **kw) == 1
        assert b"workspace" in lib.moe_last_error()
    # without groups it is attention, and so is its workspace
    assert lib.paged_attention_shared_workspace(c, b, 8, 0, 1, 0, 0, 65536, ctypes.byref(n)) == 0
    assert lib.paged_attention_workspace(c, b, 8, 0, 1, 65536, ctypes.byref(plain)) == 0
    assert n.value == plain.value
    assert lib.paged_attention_shared_workspace(c, b, 8, 1, 0, 0, 0, 0, None) == 1
    for bad in ((-1, 0, 0, 0, 0), (1, -1, 0, 0, 0), (1, 0, -1, 0, 0), (1, 0, 0, -1, 0), (1, 0, 0, 0, -1)):
        assert lib.paged_attention_shared_workspace(c, b, 8, *bad, ctypes.byref(n)) == 1


def test_empty_batches_are_no_ops(lib):  # noqa: F811
    assert _attend(lib, b=_batch(T=0)) == 0
    assert _attend(lib, b=_batch(N=0, table=None, cu_q=None, kv_len=None)) == 0
    assert _attend(lib, b=_batch(T=0), q=None, o=None, cu_group=None, shared=None, ws=None) == 0
