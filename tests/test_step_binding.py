"""The binding of include/step.h, and of attention over shared keys, where a call must not
reach the library: no GPU.  Tensors on a GPU are stood in for by torch's fake ones."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_moe_bit_gb300 as M
from sparse_moe_bit_gb300 import paged, step

BF, HF, FP, E8, I8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int8


class _Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


class _Stream:
    cuda_stream = 0x77


@pytest.fixture
def lib(monkeypatch):
    lib = _Library()
    for m in (paged, step):
        monkeypatch.setattr(m, "_library", lambda: lib)
    monkeypatch.setattr(paged, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(paged, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda self: 0x10000)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: _Stream())
    with FakeTensorMode():
        yield lib


def _e(*shape, dt=BF, dev="cuda:0"):
    return torch.empty(shape, dtype=dt, device=dev)


def _calls(dev):
    i32 = lambda *s: _e(*s, dt=torch.int32, dev=dev)
    f32 = lambda *s: _e(*s, dt=FP, dev=dev)
    bf = lambda *s: _e(*s, dev=dev)
    k, v, t, cu, n = bf(6, 16, 2, 64), bf(6, 16, 2, 64), i32(2, 4), i32(3), i32(2)
    return [
        (M.rms_norm, dict(x=bf(3, 64), weight=bf(64), residual=bf(3, 64), out=bf(3, 64), sum_out=bf(3, 64)), {}),
        (M.linear4, dict(x=_e(3, 128, dt=I8, dev=dev), codes=_e(5, 64, dt=torch.uint8, dev=dev),
                         scale=_e(5, 2, dt=HF, dev=dev), bias=_e(5, 2, dt=HF, dev=dev), x_scale=f32(3, 1),
                         out=bf(3, 5)), {}),
        (M.sample, dict(logits=f32(3, 50), u=f32(3), temperature=f32(3), top_k=i32(3), top_p=f32(3), min_p=f32(3),
                        out=i32(3)), {}),
        (M.paged_attention_shared, dict(q=bf(3, 4, 64), k_pages=k, v_pages=v, table=t, cu_q=cu, kv_len=n,
                                        cu_group=i32(2), shared=i32(1), out=bf(3, 4, 64),
                                        workspace=_e(1 << 20, dt=torch.uint8, dev=dev)), {}),
    ]


@pytest.mark.parametrize("stream", [None, _Stream()], ids=["current", "given"])
@pytest.mark.parametrize("i", range(4))
def test_tensors_elsewhere_are_refused(lib, i, stream, monkeypatch):
    monkeypatch.setattr(paged, "_have_gpu", lambda: True, raising=False)
    fn, tensors, rest = _calls("cuda:0")[i]
    fn(**tensors, **rest, stream=stream)
    assert len(lib.calls) == 1
    for where in ("cpu", "cuda:1"):
        for name in tensors:
            other = _calls(where)[i][1][name]
            with pytest.raises(ValueError):
                fn(**{**tensors, name: other}, **rest, stream=stream)
    assert len(lib.calls) == 1


def test_norm_refusals(lib):
    x, w, r = _e(3, 64), _e(64), _e(3, 64)
    for kw in (dict(x=_e(64)), dict(x=_e(2, 3, 4, 64)), dict(x=_e(3, 64, dt=E8)), dict(x=_e(64, 3).t()),
               dict(weight=_e(63)), dict(weight=_e(1, 64)), dict(weight=_e(128)[::2]), dict(residual=_e(3, 63)),
               dict(residual=_e(3, 64, dt=HF)), dict(residual=r, sum_out=_e(3, 64, dt=FP)), dict(sum_out=_e(3, 64)),
               dict(residual=r, sum_out=_e(2, 64)), dict(out=_e(3, 65)), dict(out=_e(64, 3).t()),
               dict(out=_e(3, 64), out_dtype=FP), dict(out_dtype=E8, group=48), dict(out_dtype=I8, group=-64)):
        with pytest.raises(ValueError):
            M.rms_norm(**{**dict(x=x, weight=w), **kw})
    assert lib.calls == []
    y = M.rms_norm(x, w)
    assert y.shape == (3, 64) and y.dtype is BF
    y, s, h = M.rms_norm(x, w, residual=r, out_dtype=E8, group=16)
    assert y.dtype is E8 and s.shape == (3, 4) and s.dtype is FP and h.dtype is BF
    y, s = M.rms_norm(_e(3, 5, 64)[:, 1:4], out_dtype=I8)
    assert y.shape == (3, 3, 64) and y.is_contiguous() and s.shape == (3, 3, 1)
    assert lib.calls[-1][1][1:7] == (1, 3, 3, 64, 320, 64)


def test_linear4_refusals(lib):
    x, c, s = _e(3, 128), _e(5, 64, dt=torch.uint8), _e(5, 2, dt=HF)
    x8, xs = _e(3, 128, dt=E8), _e(3, 2, dt=FP)
    for kw in (dict(x=_e(128)), dict(x=_e(3, 126)), dict(x=_e(128, 3).t()), dict(codes=_e(5, 64, dt=I8)),
               dict(codes=_e(5, 65, dt=torch.uint8)), dict(codes=_e(64, 5, dt=torch.uint8).t()),
               dict(scale=_e(4, 2, dt=HF)), dict(scale=_e(5, 3, dt=HF), bias=_e(5, 3, dt=HF)), dict(bias=_e(5, 2)),
               dict(scale=_e(5, 2, dt=FP), bias=_e(5, 2, dt=FP)), dict(scale=_e(5, 0, dt=HF), bias=_e(5, 0, dt=HF)),
               dict(bias=_e(2, 5, dt=HF).t()), dict(x_scale=xs), dict(x=x8), dict(x=x8, x_scale=_e(3, 2, dt=HF)),
               dict(x=x8, x_scale=_e(2, 2, dt=FP)), dict(x=x8, x_scale=_e(3, 3, dt=FP)),
               dict(x=x8, x_scale=_e(3, 0, dt=FP)), dict(x=x8, x_scale=_e(2, 3, dt=FP).t()), dict(out=_e(3, 6)),
               dict(out=_e(5, 3).t()), dict(out=_e(3, 5), out_dtype=FP)):
        with pytest.raises(ValueError):
            M.linear4(**{**dict(x=x, codes=c, scale=s, bias=s), **kw})
    assert lib.calls == []
    assert M.linear4(x, c, s, s).dtype is BF and M.linear4(x8, c, s, s, x_scale=xs).dtype is BF
    assert M.linear4(x, c, s, s, out_dtype=FP).dtype is FP
    assert M.linear4(x, _e(0, 64, dt=torch.uint8), _e(0, 2, dt=HF), _e(0, 2, dt=HF)).shape == (3, 0)


def test_sample_refusals(lib):
    z, u, i = _e(3, 50, dt=FP), _e(3, dt=FP), _e(3, dt=torch.int32)
    for kw in (dict(logits=_e(50, dt=FP)), dict(logits=_e(50, 3, dt=FP).t()), dict(u=_e(2, dt=FP)), dict(u=_e(3)),
               dict(u=_e(6, dt=FP)[::2]), dict(temperature=_e(3)), dict(temperature=_e(2, dt=FP)), dict(top_k=u),
               dict(top_k=_e(3, 1, dt=torch.int32)), dict(top_p=i), dict(min_p=_e(6, dt=FP)[::2]), dict(out=u),
               dict(out=_e(2, dt=torch.int32))):
        with pytest.raises(ValueError):
            M.sample(**{**dict(logits=z, u=u), **kw})
    assert lib.calls == []
    M.sample(z, u, 0.5, 10 ** 12, 0.25, 0.125)
    assert lib.calls[-1][1][6:14] == (None, None, None, None, 0.5, 0x7fffffff, 0.25, 0.125)
    t, l = M.sample(z, u, top_k=i, return_logprobs=True)
    assert t.dtype is torch.int32 and l.dtype is FP and lib.calls[-1][1][6:10] == (None, 0x10000, None, None)


def test_shared_attention_refusals(lib):
    fn, a, _ = _calls("cuda:0")[3]
    i32 = lambda *s: _e(*s, dt=torch.int32)
    for kw in (dict(cu_group=i32(3)), dict(shared=i32(1, 1)), dict(shared=_e(1, dt=FP)), dict(q=_e(3, 4, 128)),
               dict(q=_e(3, 4, 64, dt=HF)), dict(out=_e(3, 4, 64, dt=HF)), dict(out=_e(3, 3, 64)),
               dict(cu_q=i32(2)), dict(kv_len=i32(3)), dict(workspace=_e(64, 64, dt=torch.uint8).t())):
        with pytest.raises(ValueError):
            fn(**{**a, **kw})
    assert lib.calls == []
