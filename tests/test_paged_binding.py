"""The binding of include/paged.h where a call must not reach the library: no
GPU.  Tensors on a GPU are stood in for by torch's fake ones."""
import contextlib
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_moe_bit_gb300 as M
from sparse_moe_bit_gb300 import paged

BF = torch.bfloat16


class _Library:
    """Takes every call and notes its name."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


class _Stream:
    cuda_stream = 0x77


@pytest.fixture
def lib(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(paged, "_library", lambda: lib)
    monkeypatch.setattr(paged, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(paged, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda self: 0x10000)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: None)
    return lib


def _calls(dev):
    """Every call as (function, its tensors by name, what else it takes)."""
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=dev)
    bf = lambda *s: torch.empty(s, dtype=BF, device=dev)
    f = torch.empty(8, dtype=torch.float64, device=dev)
    k, v, t, cu, n = bf(6, 16, 2, 64), bf(6, 16, 2, 64), i32(1, 4), i32(2), i32(1)
    refs, lens = i32(6), i32(1)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    return [
        (M.rope, dict(x=bf(3, 4, 64), positions=i32(3), freq=f, out=bf(3, 4, 64)), {}),
        (M.rope_append, dict(q=bf(3, 4, 64), k=bf(3, 2, 64), v=bf(3, 2, 64), k_pages=k, v_pages=v,
                             table=t, cu_q=cu, kv_len=n, freq=f, q_out=bf(3, 4, 64)), {}),
        (M.paged_attention, dict(q=bf(3, 4, 64), k_pages=k, v_pages=v, table=t, cu_q=cu, kv_len=n,
                                 out=bf(3, 4, 64), workspace=ws), {}),
        (M.pages_fork, dict(refs=refs, table=t, lens=lens, src=i32(2), dst=i32(2), refused=i32(1)), {}),
        (M.pages_reserve, dict(refs=refs, table=t, lens=lens, add=i32(1)), dict(page=16)),
        (M.pages_free, dict(refs=refs, table=t, lens=lens, slots=i32(1)), {}),
        (M.pages_compact, dict(refs=refs, table=t), {}),
        (M.pages_copy, dict(pools=bf(2, 6, 16, 2, 64), moves=i32(4, 2), count=i32()), {}),
    ]


@pytest.mark.parametrize("stream", [None, _Stream()], ids=["current", "given"])
@pytest.mark.parametrize("i", range(8))
def test_tensors_elsewhere_are_refused(lib, i, stream, monkeypatch):
    """Each tensor in turn on the host, where a kernel cannot read, or on another
    device than the one that the kernels run on: an error, and no call."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: _Stream())
    monkeypatch.setattr(paged, "_have_gpu", lambda: True, raising=False)
    with FakeTensorMode():
        fn, tensors, more = _calls("cuda")[i]
        for place in ("cpu", "cuda:1"):
            for name, t in tensors.items():
                other = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=place)
                with pytest.raises(ValueError):
                    fn(**dict(tensors, **{name: other}), **more, stream=stream)
            elsewhere = {n: torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=place)
                         for n, t in tensors.items()}
            with pytest.raises(ValueError):
                fn(**elsewhere, **more, stream=stream)
        assert lib.calls == []
        fn(**tensors, **more, stream=stream)
        assert lib.calls


def test_buffers_smaller_than_what_is_written_are_refused(lib):
    """A workspace whose elements share memory, and counts that are not one int32:
    the library would read and write past them."""
    with FakeTensorMode():
        calls = _calls("cuda")
        one = torch.empty(1, dtype=torch.uint8, device="cuda")
        wide = torch.empty(1 << 20, 2, dtype=torch.uint8, device="cuda")
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
        for i, name, bad in [(2, "workspace", one.expand(1 << 20)), (2, "workspace", wide[:, 0]),
                             (3, "refused", i32(1).to(torch.uint8)), (3, "refused", i32(0)),
                             (3, "refused", i32(2)), (7, "count", i32(0)), (7, "count", i32(3)),
                             (7, "count", i32(1).long())]:
            fn, tensors, more = calls[i]
            with pytest.raises(ValueError):
                fn(**dict(tensors, **{name: bad}), **more)
        assert lib.calls == []
        for i, name, good in [(3, "refused", i32()), (7, "count", i32(1)), (7, "count", None),
                              (2, "workspace", torch.empty(64, 64, device="cuda"))]:
            fn, tensors, more = calls[i]
            fn(**dict(tensors, **{name: good}), **more)


class _Pool:
    """Stands in for the streams of torch: which one is current, and which one each
    tensor was made on and is said to be used on."""

    def __init__(self, monkeypatch):
        self.current, self.made, self.told = "mine", {}, {}
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw: raw)
        monkeypatch.setattr(torch.cuda, "stream", self._enter)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: self.told.setdefault(id(t), []).append(s))
        for name in ("empty", "empty_strided"):
            monkeypatch.setattr(torch, name, self._maker(getattr(torch, name)))
        self.kept = []

    @contextlib.contextmanager
    def _enter(self, stream):
        old, self.current = self.current, stream
        yield
        self.current = old

    def _maker(self, make):
        def f(*args, **kw):
            t = make(*args, **kw)
            if sys._getframe(1).f_globals["__name__"] == paged.__name__:
                self.made[id(t)] = self.current
                self.kept.append(t)
            return t
        return f


@pytest.mark.parametrize("given", [False, True], ids=["made", "given"])
@pytest.mark.parametrize("i", range(8))
def test_tensors_come_from_the_pool_of_the_stream_that_writes_them(lib, monkeypatch, i, given):
    """What a call makes for a given stream to write must not be a block that the
    current stream may still be using; what it returns is used on the current
    stream, and what it was given to write on the given one."""
    with FakeTensorMode():
        fn, tensors, more = _calls("cuda")[i]
        if not given:
            tensors = {n: t for n, t in tensors.items()
                       if n not in ("out", "q_out", "workspace", "refused", "count")}
        if fn is M.paged_attention:
            more = dict(return_lse=True)
            monkeypatch.setattr(paged, "_sizes", _Sizes())
        pool = _Pool(monkeypatch)
        r = fn(**tensors, **more, stream=_Stream())
        assert [s for s in pool.made.values() if s != 0x77] == []
        mine = [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]
        for t in mine:
            if id(t) in pool.made:
                assert pool.told.get(id(t)) == ["mine"]
        for n in ("out", "q_out", "workspace"):
            if n in tensors:
                assert pool.told.get(id(tensors[n])) == [0x77]


class _Sizes(dict):
    """Every call needs a workspace."""

    def get(self, key):
        return 4096
