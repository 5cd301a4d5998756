"""A small serving loop over the framework's layers: attention over a paged
cache next to the MoE block.

A prompt is read in chunks, forked into continuations that share its pages,
decoded step by step (the shared last page is copied when a continuation first
writes to it), the finished continuations give their pages back, the cache is
compacted, and the survivors go on.  ``python examples/serve.py`` runs it on
random weights and prints how far a continuation decoded this way is from the
same tokens read as one prompt.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_moe_bit_gb300 as M  # noqa: E402
from synth import device as sd  # noqa: E402
from synth import gen  # noqa: E402


@dataclass
class Shape:
    layers: int = 2
    d: int = 256       # hidden size
    hq: int = 8        # query heads
    hk: int = 2        # key/value heads
    dim: int = 64      # features of a head
    rotary: int = 32   # of which turn
    page: int = 16
    pages: int = 64
    slots: int = 8
    width: int = 16    # pages of a slot, at most


class Server:
    """Weights, cache and page state; ``step`` runs new tokens of some slots."""

    def __init__(self, s: Shape, seed: int = 0):
        self.s = s
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *n: (torch.randn(*n, device="cuda", generator=g) * n[0] ** -0.5).bfloat16()
        self.w_qkv = [rand(s.d, (s.hq + 2 * s.hk) * s.dim) for _ in range(s.layers)]
        self.w_out = [rand(s.hq * s.dim, s.d) for _ in range(s.layers)]
        shape = gen.MoEShape(d=s.d, E=16, k=2, I=128)
        self.moe = [M.MoE(M.MoEConfig(d=s.d, E=16, k=2, I=128, max_tokens=256),
                          sd.host_layer_to_device(gen.make_layer(seed, i, shape)))
                    for i in range(s.layers)]
        self.freq, self.mscale = M.rope_frequencies(s.rotary, 1e6, "yarn", factor=4.0, original=64,
                                                    device="cuda")
        # all layers' keys and values in one array: one call copies a page of them all
        self.cache = torch.zeros(s.layers * 2, s.pages, s.page, s.hk, s.dim, dtype=torch.bfloat16,
                                 device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(s.pages, **i32)
        self.table = torch.full((s.slots, s.width), -1, **i32)
        self.lens = torch.zeros(s.slots, **i32)
        self.held = [0] * s.slots   # the host's copy of lens: it hands out the work

    def step(self, slots: list, xs: list) -> list:
        """New tokens xs[i] [n, d] of slot slots[i], all slots in one pass; returns
        their hidden states behind the last layer."""
        s = self.s
        add = [0] * s.slots
        for i, x in zip(slots, xs):
            add[i] += x.shape[0]
            self.held[i] += x.shape[0]
        moves, status = M.pages_reserve(self.refs, self.table, self.lens,
                                        torch.tensor(add, dtype=torch.int32, device="cuda"), s.page)
        if status.tolist() != [0, 0]:
            raise RuntimeError("the cache is full")
        M.pages_copy(self.cache, moves)
        new = [x.shape[0] for x in xs]
        cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        rows = torch.tensor(slots, device="cuda")
        table, kv_len = self.table[rows], self.lens[rows]
        hints = dict(max_q=max(new), max_kv=max(self.held[i] for i in slots))
        x = torch.cat(xs)
        for l in range(s.layers):
            qkv = (_rms(x) @ self.w_qkv[l]).view(-1, s.hq + 2 * s.hk, s.dim)
            q, k, v = qkv.split([s.hq, s.hk, s.hk], 1)
            kp, vp = self.cache[2 * l], self.cache[2 * l + 1]
            q = M.rope_append(q, k, v, kp, vp, table, cu, kv_len, self.freq, mscale=self.mscale)
            o = M.paged_attention(q, kp, vp, table, cu, kv_len, **hints)
            x = x + o.view(-1, s.hq * s.dim) @ self.w_out[l]
            x = x + self.moe[l].forward(_rms(x))
        return list(x.split(new))

    def fork(self, src: int, dst: list):
        i32 = dict(dtype=torch.int32, device="cuda")
        M.pages_fork(self.refs, self.table, self.lens, torch.full((len(dst),), src, **i32),
                     torch.tensor(dst, **i32))
        for i in dst:
            self.held[i] = self.held[src]

    def release(self, slots: list):
        M.pages_free(self.refs, self.table, self.lens,
                     torch.tensor(slots, dtype=torch.int32, device="cuda"))
        for i in slots:
            self.held[i] = 0
        moves, count = M.pages_compact(self.refs, self.table)
        M.pages_copy(self.cache, moves, count)

    def pages_in_use(self) -> int:
        return int((self.refs > 0).sum())


def _rms(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def run(seed: int = 0):
    """The loop; returns (relative error of the decoded continuation against the
    same tokens read as one prompt, pages in use before and after compaction)."""
    s = Shape()
    srv = Server(s, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    toks = lambda n: torch.randn(n, s.d, device="cuda", generator=g).bfloat16()
    prompt, tails = toks(75), [toks(9) for _ in range(3)]
    for a, b in ((0, 40), (40, 75)):                  # the prompt, in chunks
        srv.step([0], [prompt[a:b]])
    srv.fork(0, [1, 2, 3])
    for i in range(4):                                # three continuations, token by token
        srv.step([1, 2, 3], [t[i:i + 1] for t in tails])
    before = srv.pages_in_use()
    srv.release([0, 2])
    after = srv.pages_in_use()
    for i in range(4, 8):
        srv.step([1, 3], [tails[0][i:i + 1], tails[2][i:i + 1]])
    last = srv.step([3, 1], [tails[2][8:9], tails[0][8:9]])[0]
    whole = srv.step([5], [torch.cat([prompt, tails[2]])])[0][-1:]
    err = ((last.float() - whole.float()).norm() / whole.float().norm()).item()
    if M.paged_device_error():
        raise RuntimeError("device error")
    return err, before, after


if __name__ == "__main__":
    e, before, after = run()
    print(f"continuation against one prompt: relative error {e:.2e}; "
          f"pages in use {before} -> {after}")
