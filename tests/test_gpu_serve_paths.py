"""Which calls the serving example makes: a prompt's chunk goes through plain attention and
products of 16-bit weights, continuations of one prompt through attention over their shared keys
and 4-bit products."""
import collections
import importlib.util
import os
import sys

import pytest
import torch

import sparse_moe_bit_gb300 as M

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_of_a_step(monkeypatch):
    spec = importlib.util.spec_from_file_location("serve", os.path.join(ROOT, "examples", "serve.py"))
    m = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, "serve", m)
    spec.loader.exec_module(m)
    s = m.Shape()
    server = m.Server(s)
    calls = collections.Counter()

    def counted(name, f):
        def call(*a, **kw):
            calls[name] += 1
            return f(*a, **kw)
        return call

    names = ("paged_attention", "paged_attention_shared", "linear4")
    for n in names:
        monkeypatch.setattr(M, n, counted(n, getattr(M, n)))

    def step(slots, lengths):
        calls.clear()
        g = torch.Generator(device="cuda").manual_seed(sum(lengths))
        server.step(slots, [torch.randint(0, s.vocab, (n,), dtype=torch.int32, device="cuda", generator=g) for n in lengths])
        return tuple(calls[n] // s.layers for n in names)

    assert step([0], [40]) == (1, 0, 0)               # a prompt's chunk
    server.fork(0, [1, 2])
    assert step([1, 2], [1, 1]) == (0, 1, 2)          # its continuations
    assert step([0, 1, 2, 5], [1, 1, 1, 30]) == (0, 1, 0)   # and beside another prompt
    assert step([1], [1]) == (1, 0, 2)                # one of them alone
    torch.cuda.synchronize()
    assert M.paged_device_error() == 0
