"""include/paged.h: exports, refusals of bad arguments (before anything could
be enqueued), and the host-side frequency tables.  No GPU."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_A = 0x10000  # a fake, aligned device address: only ever checked


@pytest.fixture(scope="module")
def lib():
    from sparse_moe_bit_gb300 import build, moe, paged
    if not os.path.exists(moe.LIB_PATH):
        build.build()
    return paged._library()


def test_header_and_binding_agree(lib):
    from sparse_moe_bit_gb300 import paged
    src = open(os.path.join(ROOT, "include", "paged.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"\bmoe_status\s+([a-z_]+)\s*\(", src)
    assert sorted(names) == sorted(paged.EXPORTS)
    for n in names:
        assert hasattr(lib, n)


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("pages", ctypes.c_int), ("page", ctypes.c_int), ("heads", ctypes.c_int),
                ("dim", ctypes.c_int), ("page_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Batch(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("N", ctypes.c_int), ("T", ctypes.c_int),
                ("width", ctypes.c_int), ("table_stride", ctypes.c_int64)]


def test_binding_packs_the_structures(lib):
    from sparse_moe_bit_gb300 import paged
    assert paged._CACHE.size == ctypes.sizeof(_Cache) and paged._BATCH.size == ctypes.sizeof(_Batch)
    c = _Cache.from_buffer_copy(paged._CACHE.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 10))
    assert [getattr(c, n) for n, _ in _Cache._fields_] == list(range(1, 11))
    b = _Batch.from_buffer_copy(paged._BATCH.pack(1, 2, 3, 4, 5, 6, 7))
    assert [getattr(b, n) for n, _ in _Batch._fields_] == list(range(1, 8))


def _cache(**kw):
    a = dict(k=_A, v=_A, dtype=1, pages=8, page=16, heads=2, dim=128, page_stride=16 * 256,
             row_stride=256, head_stride=128)
    a.update(kw)
    return bytes(_Cache(**a))


def _batch(**kw):
    a = dict(table=_A, cu_q=_A, kv_len=_A, N=2, T=4, width=4, table_stride=4)
    a.update(kw)
    return bytes(_Batch(**a))


CACHE_BAD = [(dict(k=None), 1), (dict(v=_A + 8), 1), (dict(dtype=3), 1), (dict(dtype=0), 1),
             (dict(pages=0), 1), (dict(page=0), 1), (dict(heads=0), 1), (dict(row_stride=252), 1),
             (dict(page_stride=-8), 1), (dict(dim=96), 2), (dict(dim=512), 2)]
BATCH_BAD = [(dict(N=-1), 1), (dict(T=-1), 1), (dict(width=-1), 1), (dict(table=None), 1),
             (dict(cu_q=None), 1), (dict(kv_len=_A + 2), 1)]


def _attend(lib, c=None, b=None, **kw):
    a = dict(q=_A, q_ts=1024, q_hs=128, Hq=8, scale=0.1, causal=1, window=0, max_q=1, max_kv=64,
             o=_A, o_ts=1024, o_hs=128, lse=None, ws=None, ws_bytes=0)
    a.update(kw)
    c, b = c or _cache(), b or _batch()
    return lib.paged_attention(a["q"], a["q_ts"], a["q_hs"], a["Hq"], c,
                               b, a["scale"], a["causal"], a["window"], a["max_q"],
                               a["max_kv"], a["o"], a["o_ts"], a["o_hs"], a["lse"], a["ws"],
                               a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(q=_A + 8), 1), (dict(q_ts=1020), 1),
    (dict(o_hs=-128), 1), (dict(Hq=0), 1), (dict(Hq=7), 1), (dict(scale=0.0), 1),
    (dict(scale=-0.1), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(window=-1), 1), (dict(max_q=-1), 1), (dict(max_kv=-2), 1), (dict(lse=_A + 2), 1),
    (dict(ws=_A + 8), 1)])
def test_attention_rejects_bad_arguments(lib, kw, status):
    assert _attend(lib, **kw) == status, lib.moe_last_error()
    assert lib.moe_last_error()


@pytest.mark.parametrize("kw,status", CACHE_BAD)
def test_bad_cache_is_rejected(lib, kw, status):
    assert _attend(lib, c=_cache(**kw)) == status
    n = ctypes.c_size_t()
    c, b = _cache(**kw), _batch()
    assert lib.paged_attention_workspace(c, b, 8, 0, 1, 64,
                                         ctypes.byref(n)) == status
    assert lib.rope_append(_A, 1024, _A, 8, _A, 256, _A, 256, c, b, _A,
                           16, 1.0, 0, None) == status


@pytest.mark.parametrize("kw,status", BATCH_BAD)
def test_bad_batch_is_rejected(lib, kw, status):
    assert _attend(lib, b=_batch(**kw)) == status


def test_attention_needs_its_workspace(lib):
    """A long context on few rows is split over the keys: the call without the
    workspace that the split needs is refused."""
    c, b = _cache(pages=4096), _batch(N=1, T=1, width=4096, table_stride=4096)
    n = ctypes.c_size_t()
    assert lib.paged_attention_workspace(c, b, 8, 0, 1, 65536,
                                         ctypes.byref(n)) == 0
    assert n.value > 0
    assert _attend(lib, c=c, b=b, max_kv=65536, ws=_A, ws_bytes=n.value - 1) == 1
    assert b"workspace" in lib.moe_last_error()
    assert _attend(lib, c=c, b=b, max_kv=65536) == 1


def test_empty_batches_are_no_ops(lib):
    assert _attend(lib, b=_batch(T=0)) == 0
    assert _attend(lib, b=_batch(N=0, table=None, cu_q=None, kv_len=None)) == 0
    assert _attend(lib, b=_batch(T=0), q=None, o=None) == 0
    c, b = _cache(), _batch(T=0)
    assert lib.rope_append(None, 0, None, 8, None, 0, None, 0, c, b,
                           _A, 16, 1.0, 0, None) == 0
    assert lib.rope(None, None, 1, 0, 4, 64, 256, 64, 256, 64, None, _A, 8, 1.0, 0, 0, None) == 0
    assert lib.pages_copy(None, 0, 0, 4, 64, 64, None, 0, None, None) == 0
    assert lib.pages_free(_A, 4, _A, 4, 4, _A, 2, None, 0, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(pos=None), 1), (dict(dtype=0), 1),
    (dict(dtype=4), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(D=0), 1), (dict(r=0), 1),
    (dict(r=33), 1), (dict(D=2048), 1), (dict(freq=None), 1), (dict(freq=_A + 4), 1),
    (dict(mscale=math.nan), 1), (dict(x=_A + 1), 1), (dict(pos=_A + 2), 1),
    (dict(x=_A, out=_A, o_ts=512), 1), (dict(H=1 << 20), 2)])
def test_rope_rejects_bad_arguments(lib, kw, status):
    a = dict(x=_A, out=2 * _A, dtype=1, T=3, H=4, D=64, x_ts=256, x_hs=64, o_ts=256, o_hs=64,
             pos=_A, freq=_A, r=16, mscale=1.0)
    a.update(kw)
    r = lib.rope(a["x"], a["out"], a["dtype"], a["T"], a["H"], a["D"], a["x_ts"], a["x_hs"],
                 a["o_ts"], a["o_hs"], a["pos"], a["freq"], a["r"], a["mscale"], 0, 0, None)
    assert r == status, lib.moe_last_error()
    assert lib.moe_last_error()


@pytest.mark.parametrize("kw", [dict(q=None), dict(q_out=None), dict(k=None), dict(v=None),
                                dict(Hq=0), dict(r=65), dict(freq=None), dict(mscale=math.inf),
                                dict(k=_A + 1), dict(q_out=_A, q_ts=2048)])
def test_append_rejects_bad_arguments(lib, kw):
    a = dict(q=_A, q_ts=1024, q_out=2 * _A, Hq=8, k=_A, v=_A, freq=_A, r=16, mscale=1.0)
    a.update(kw)
    c, b = _cache(), _batch()
    assert lib.rope_append(a["q"], a["q_ts"], a["q_out"], a["Hq"], a["k"], 256, a["v"], 256,
                           c, b, a["freq"], a["r"], a["mscale"], 0,
                           None) == 1


@pytest.mark.parametrize("call", [
    lambda L: L.pages_fork(None, 4, _A, 4, 4, _A, 2, _A, _A, 1, None, None),
    lambda L: L.pages_fork(_A, 0, _A, 4, 4, _A, 2, _A, _A, 1, None, None),
    lambda L: L.pages_fork(_A, 4, _A, 3, 4, _A, 2, _A, _A, 1, None, None),
    lambda L: L.pages_fork(_A, 4, _A, 4, 4, _A, 2, None, _A, 1, None, None),
    lambda L: L.pages_fork(_A, 4, _A, 4, 4, _A, 2, _A, _A, -1, None, None),
    lambda L: L.pages_fork(_A, 4, _A, 4, 4, _A, 2, _A, _A, 1, _A + 1, None),
    lambda L: L.pages_reserve(_A, 4, _A, 4, 4, _A, _A, 2, 0, _A, _A, _A, None),
    lambda L: L.pages_reserve(_A, 4, _A, 4, 4, _A, None, 2, 16, _A, _A, _A, None),
    lambda L: L.pages_reserve(_A, 4, _A, 4, 4, _A, _A, 2, 16, _A, None, _A, None),
    lambda L: L.pages_reserve(_A, 4, _A, 4, 4, _A, _A, 2, 16, _A, _A, _A + 2, None),
    lambda L: L.pages_free(_A, 4, _A, 4, 4, None, 2, _A, 1, None),
    lambda L: L.pages_free(_A, 4, _A, 4, 4, _A, 2, None, 1, None),
    lambda L: L.pages_compact(_A, 4, _A, 4, 4, 2, None, _A, _A, None),
    lambda L: L.pages_compact(_A, 4, _A, 4, -1, 2, _A, _A, _A, None),
    lambda L: L.pages_copy(_A, 2, 4096, 4, 1024, 1000, _A, 1, None, None),
    lambda L: L.pages_copy(_A, 2, 4096, 4, 512, 1024, _A, 1, None, None),
    lambda L: L.pages_copy(_A + 8, 2, 4096, 4, 1024, 1024, _A, 1, None, None),
    lambda L: L.pages_copy(_A, 2, 4096, 4, 1024, 1024, None, 1, None, None),
    lambda L: L.paged_get_device_error(None, None)])
def test_page_calls_reject_bad_arguments(lib, call):
    assert call(lib) == 1
    assert lib.moe_last_error()


def test_oversized_page_state_is_unsupported(lib):
    assert lib.pages_free(_A, 4, _A, 1 << 16, 1 << 16, _A, 1 << 15, _A, 1, None) == 2


def test_binding_checks_shapes_and_types():
    import sparse_moe_bit_gb300 as M
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    t, cu, n = (torch.zeros(s, dtype=torch.int32) for s in ((1, 2), (2,), (1,)))
    bad = [dict(q=q.half()), dict(k=k.half()), dict(k=k.transpose(1, 2)), dict(t=t.long()),
           dict(cu=cu[:1]), dict(n=n.float()), dict(k=k[..., :32])]
    for kw in bad:
        a = dict(q=q, k=k, v=k, t=t, cu=cu, n=n)
        a.update(kw)
        with pytest.raises(ValueError):
            M.paged_attention(a["q"], a["k"], a["v"], a["t"], a["cu"], a["n"])
    f = torch.ones(8, dtype=torch.float64)
    pos = torch.zeros(2, dtype=torch.int32)
    for args in ((q[0], pos, f), (q, pos.long(), f), (q, pos[:1], f), (q, pos, f.float()),
                 (q.double(), pos, f), (q.transpose(1, 2), pos, f)):
        with pytest.raises(ValueError):
            M.rope(*args)
    with pytest.raises(ValueError):
        M.rope_append(q, k[:2, 0], k[:2, 0].half(), k, k, t, cu, n, f)
    with pytest.raises(ValueError):
        M.pages_copy(k.transpose(1, 2)[None], torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        M.pages_fork(n, t, n, n.long(), n)
    with pytest.raises(ValueError):
        M.rope_frequencies(64, scaling="other")


# ----------------------------------------------------------- frequency tables
def test_plain_linear_and_ntk_frequencies():
    import sparse_moe_bit_gb300 as M
    f, m = M.rope_frequencies(64, 10000.0)
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert f.dtype is torch.float64 and m == 1.0
    np.testing.assert_allclose(f.numpy(), want, rtol=1e-14)
    f, m = M.rope_frequencies(64, 10000.0, "linear", factor=4.0)
    np.testing.assert_allclose(f.numpy(), np.array(want) / 4, rtol=1e-14)
    f, m = M.rope_frequencies(64, 10000.0, "ntk", factor=4.0)
    # the fastest pair keeps its speed, the slowest is slowed by the factor
    assert f[0] == 1.0 and m == 1.0
    np.testing.assert_allclose(f[-1].item(), want[-1] / 4, rtol=1e-12)


def test_yarn_and_banded_frequencies_keep_fast_pairs_and_slow_slow_ones():
    import sparse_moe_bit_gb300 as M
    base = np.array([500000.0 ** (-2 * i / 128) for i in range(64)])
    f, m = M.rope_frequencies(128, 500000.0, "yarn", factor=8.0, original=32768, low=1.0, high=32.0)
    assert abs(m - (0.1 * math.log(8.0) + 1.0)) < 1e-15
    turns = 32768 * base / (2 * math.pi)
    fast, slow = turns > 34, turns < 0.9   # clear of the rounded ends of the ramp
    fast[np.argmin(fast):] = False
    np.testing.assert_allclose(f.numpy()[:np.sum(turns > 60)], base[:np.sum(turns > 60)], rtol=1e-14)
    np.testing.assert_allclose(f.numpy()[turns < 0.6], base[turns < 0.6] / 8, rtol=1e-14)
    assert np.all(np.diff(f.numpy()) < 0)
    f, m = M.rope_frequencies(128, 500000.0, "banded", factor=8.0, original=8192, low=1.0, high=4.0)
    turns = 8192 * base / (2 * math.pi)
    assert m == 1.0
    np.testing.assert_allclose(f.numpy()[turns >= 4], base[turns >= 4], rtol=1e-14)
    np.testing.assert_allclose(f.numpy()[turns <= 1], base[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    s = (turns[mid] - 1) / 3
    np.testing.assert_allclose(f.numpy()[mid], base[mid] * (s + (1 - s) / 8), rtol=1e-13)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(base=0.0), dict(base=-1.0), dict(base=math.inf),
    dict(scaling="linear", factor=0.0), dict(scaling="ntk", rotary_dim=2, factor=2.0),
    dict(scaling="yarn", factor=2.0, original=0), dict(scaling="banded", factor=2.0, original=64, low=4.0, high=1.0),
    dict(scaling="yarn", factor=2.0, original=64, base=1.0)])
def test_frequency_refusals(kw):
    import sparse_moe_bit_gb300 as M
    a = dict(rotary_dim=64)
    a.update(kw)
    with pytest.raises(M.MoEError) as ex:
        M.rope_frequencies(a.pop("rotary_dim"), **a)
    assert ex.value.status == 1


def test_calls_fail_loudly_without_a_device():
    """With no device a valid call passes the checks and then raises: there is
    no CPU fallback.  Skipped where a device exists (the tensors live here)."""
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    import types
    import sparse_moe_bit_gb300 as M
    legacy = types.SimpleNamespace(cuda_stream=0)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    f = torch.ones(8, dtype=torch.float64)
    for call in (lambda: M.paged_attention(q, k, k, t, cu, n, max_kv=16, stream=legacy),
                 lambda: M.rope(q, n, f, stream=legacy),
                 lambda: M.rope_append(q, k[:1, 0], k[:1, 0], k, k, t, cu, n, f, stream=legacy),
                 lambda: M.pages_compact(n, t, stream=legacy)):
        with pytest.raises(M.MoEError) as ex:
            call()
        assert ex.value.status == 3
