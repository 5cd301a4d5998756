"""include/step.h: exports, refusals of bad arguments before anything could be
enqueued, and the definitions' own pins.  No GPU."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

from oracle import step_oracle as SO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_A = 0x10000  # fake, aligned device addresses: only ever checked
_B, _C, _D = 0x20000, 0x30000, 0x40000


@pytest.fixture(scope="module")
def lib():
    from sparse_moe_bit_gb300 import build, moe, step
    if not os.path.exists(moe.LIB_PATH):
        build.build()
    return step._library()


def test_header_and_binding_agree(lib):
    from sparse_moe_bit_gb300 import step
    src = open(os.path.join(ROOT, "include", "step.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"\bmoe_status\s+([a-z_0-9]+)\s*\(", src)
    assert sorted(names) == sorted(step.EXPORTS)
    for n in names:
        assert hasattr(lib, n)


def _norm(lib, **kw):
    a = dict(x=_A, dtype=1, T=4, H=2, d=64, x_ts=128, x_hs=64, r=_B, r_ts=128, r_hs=64, s=_C, s_ts=128,
             s_hs=64, w=_D, w_dtype=1, unit=0, eps=1e-6, y=0x50000, y_dtype=1, y_ts=128, y_hs=64, scales=None,
             group=0, stream=None)
    a.update(kw)
    return lib.rms_norm(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(dtype=0), 1), (dict(dtype=4), 1), (dict(y_dtype=0), 1),
    (dict(y_dtype=6), 1), (dict(w_dtype=2), 1), (dict(w_dtype=0), 1), (dict(T=-1), 1), (dict(H=0), 1),
    (dict(d=0), 1), (dict(d=32769), 2), (dict(eps=-1e-6), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(group=32), 1), (dict(y_dtype=4, scales=_B + 0x90000, group=48), 1), (dict(y_dtype=4), 1),
    (dict(y_dtype=5, scales=_B + 0x90000, group=-1), 1), (dict(scales=_B + 0x90000), 1), (dict(r=None), 1),
    (dict(s=None), 1), (dict(x=_A + 1), 1), (dict(w=_D + 1), 1), (dict(y=_A, y_ts=256), 1),
    (dict(y=_A, y_dtype=3), 1), (dict(y=_A, s=_A), 1), (dict(y=_C), 1), (dict(y=_B), 1), (dict(s=_B, s_ts=64), 1),
    (dict(s=_A, s_hs=128), 1), (dict(T=1 << 30, H=4), 2),
    (dict(w=None, unit=1), 1), (dict(T=(1 << 31) - 4, H=1), 2)])
def test_norm_rejects_bad_arguments(lib, kw, status):
    assert _norm(lib, **kw) == status, lib.moe_last_error()
    assert lib.moe_last_error()


def _linear(lib, **kw):
    a = dict(x=_A, x_dtype=1, T=4, K=256, x_ts=256, x_scale=None, x_group=0, codes=_B, scale=_C, bias=_D,
             scale_dtype=1, O=64, group=64, y=0x50000, y_dtype=1, y_ts=64, stream=None)
    a.update(kw)
    return lib.linear4(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(codes=None), 1), (dict(scale=None), 1), (dict(bias=None), 1), (dict(y=None), 1),
    (dict(x_dtype=3), 1), (dict(x_dtype=0), 1), (dict(y_dtype=4), 1), (dict(scale_dtype=3), 1), (dict(T=-1), 1),
    (dict(K=0), 1), (dict(O=0), 1), (dict(group=96), 1), (dict(group=0), 1), (dict(group=32), 2),
    (dict(K=100, group=50), 2), (dict(x_group=64), 1), (dict(x_dtype=4), 1), (dict(x_scale=_D), 1),
    (dict(x_dtype=4, x_scale=_D, x_group=96), 1), (dict(x_dtype=5, x_scale=_D, x_group=32), 2),
    (dict(x_dtype=4, x_scale=_D + 2), 1), (dict(x=_A + 8), 1), (dict(x_ts=260), 1), (dict(codes=_B + 8), 1),
    (dict(scale=_C + 2), 1), (dict(y=0x50001), 1), (dict(K=36928), 2), (dict(O=(1 << 30) + 1), 2),
    (dict(T=524281), 2)])
def test_linear4_rejects_bad_arguments(lib, kw, status):
    assert _linear(lib, **kw) == status, lib.moe_last_error()
    assert lib.moe_last_error()


def _sample(lib, **kw):
    a = dict(logits=_A, dtype=3, B=2, V=100, stride=100, u=_B, t=_C, k=_C, p=_C, m=_C, t0=1.0, k0=0, p0=1.0, m0=0.0, token=_D, logprob=None,
             stream=None)
    a.update(kw)
    return lib.sample(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), 1), (dict(u=None), 1), (dict(token=None), 1), (dict(dtype=4), 1), (dict(dtype=0), 1),
    (dict(B=-1), 1), (dict(V=0), 1), (dict(V=360449), 2), (dict(logits=_A + 2), 1), (dict(u=_B + 2), 1),
    (dict(t=_C + 1), 1), (dict(k=_C + 1), 1), (dict(p=_C + 2), 1), (dict(m=_C + 2), 1), (dict(token=_D + 2), 1),
    (dict(logprob=_D + 2), 1)])
def test_sample_rejects_bad_arguments(lib, kw, status):
    assert _sample(lib, **kw) == status, lib.moe_last_error()
    assert lib.moe_last_error()


def test_empty_calls_are_no_ops(lib):
    assert _norm(lib, T=0) == 0 and _norm(lib, T=0, x=None, y=None) == 0
    assert _linear(lib, T=0) == 0 and _linear(lib, T=0, x=None, y=None) == 0
    assert _sample(lib, B=0) == 0 and _sample(lib, B=0, logits=None, u=None, token=None) == 0


# ---- the definitions on cases done by hand
def test_norm_definition():
    n, s = SO.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), np.array([[0.0, 0.0]]), 0.0)
    assert np.allclose(n, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]]) and np.array_equal(s, [[3.0, 4.0]])
    assert np.allclose(SO.rms_norm(np.array([[1.0, 1.0]]), np.zeros(2), offset=1.0, eps=0.0)[0], 1.0)
    assert np.allclose(SO.scales(np.array([[1.0, -448.0, 0.5, 0.25]]), 2, "e4m3"), [[1.0, 0.5 / 448]])


def test_linear4_definition():
    codes = np.array([[0x21, 0x43]], np.uint8)  # 1, 2, 3, 4
    assert np.array_equal(SO.weights4(codes, np.array([[0.5, 1.0]]), np.array([[0.0, -3.0]])),
                          [[0.5, 1.0, 0.0, 1.0]])


def test_sample_definition():
    z = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert [SO.sample(z, u)[0] for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [SO.sample(z, u, top_k=2)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert [SO.sample(z, u, top_p=0.65)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert [SO.sample(z, u, top_p=0.75)[0] for u in (0.43, 0.45, 0.66, 0.67)] == [1, 2, 2, 3]
    assert [SO.sample(z, u, min_p=0.6)[0] for u in (0.57, 0.58)] == [1, 3]
    assert SO.sample(z, 0.5, temperature=0.0) == (1, 0.0)
    assert SO.sample(np.array([1.0, 1.0, 1.0]), 0.9, top_k=2)[0] == 1           # ties: the first by index
    assert SO.sample(np.array([np.nan, -np.inf]), 0.5)[0] == -1
    assert SO.sample(np.array([0.0, np.inf, np.inf]), 0.6)[0] == 2
    assert math.isclose(SO.sample(z, 0.2, top_k=2)[1], math.log(4 / 7))
