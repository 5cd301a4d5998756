"""include/step.h: outputs whose rows would be written over one another are refused before
anything could be enqueued.  No GPU."""
import os

import pytest

_A, _R, _S, _W, _Y = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000  # fake addresses: only ever checked


@pytest.fixture(scope="module")
def lib():
    from sparse_moe_bit_gb300 import build, moe, step
    if not os.path.exists(moe.LIB_PATH):
        build.build()
    return step._library()


@pytest.mark.parametrize("kw", [dict(y_ts=0), dict(y_hs=0), dict(y_ts=63), dict(y_hs=63), dict(y_ts=-63), dict(s_ts=0),
                                dict(s_hs=0), dict(s_hs=63), dict(T=2, H=1, y_ts=0), dict(T=1, H=2, s_hs=0)])
def test_norm(lib, kw):
    a = dict(x=_A, dtype=1, T=4, H=2, d=64, x_ts=128, x_hs=64, r=_R, r_ts=128, r_hs=64, s=_S, s_ts=128,
             s_hs=64, w=_W, w_dtype=1, unit=0, eps=1e-6, y=_Y, y_dtype=1, y_ts=128, y_hs=64, scales=None,
             group=0, stream=None)
    a.update(kw)
    assert lib.rms_norm(*a.values()) == 1
    assert b"overlap" in lib.moe_last_error()


@pytest.mark.parametrize("kw", [dict(y_ts=0), dict(y_ts=63), dict(y_ts=-63), dict(T=2, y_ts=1)])
def test_linear4(lib, kw):
    a = dict(x=_A, x_dtype=1, T=4, K=256, x_ts=256, x_scale=None, x_group=0, codes=_R, scale=_S, bias=_W,
             scale_dtype=1, O=64, group=64, y=_Y, y_dtype=1, y_ts=64, stream=None)
    a.update(kw)
    assert lib.linear4(*a.values()) == 1
    assert b"overlap" in lib.moe_last_error()
