"""A small serving loop over the framework's layers: attention over a paged
cache next to the MoE block, between norms and projections with 4-bit weights.

A prompt is read in chunks and forked into continuations that share its pages.
They are decoded together, token by token: the prompt's keys are read once for
all of them, each next token is drawn from its logits, the shared last page is
copied when a continuation first writes to it.  The finished continuations give
their pages back, the cache is compacted, and the survivors go on.  ``python
examples/serve.py`` runs it on random weights and prints how far a continuation
decoded this way is from the same tokens read as one prompt.
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
    vocab: int = 1000
    page: int = 16
    pages: int = 64
    slots: int = 8
    width: int = 16    # pages of a slot, at most


class Server:
    """Weights, cache and page state; ``step`` runs new tokens of some slots."""

    def __init__(self, s: Shape, seed: int = 0):
        self.s = s
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(k, o):
            """4-bit weights of standard deviation k^-1/2, groups of 64: codes, scales, biases."""
            codes = torch.randint(0, 256, (o, k // 2), dtype=torch.uint8, device="cuda", generator=g)
            step = torch.full((o, k // 64), (12 / k) ** 0.5 / 15, dtype=torch.float16, device="cuda")
            return codes, step, -7.5 * step

        def dense(codes, step, bias):
            """The same weights in 16 bits, for the products of a prompt."""
            c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1, 64)
            return (c * step[..., None].float() + bias[..., None].float()).flatten(1).bfloat16()

        def norm():
            return (1 + 0.1 * torch.randn(s.d, device="cuda", generator=g)).bfloat16()

        self.embedding = torch.randn(s.vocab, s.d, device="cuda", generator=g).bfloat16()
        self.w_qkv = [weights(s.d, (s.hq + 2 * s.hk) * s.dim) for _ in range(s.layers)]
        self.w_out = [weights(s.hq * s.dim, s.d) for _ in range(s.layers)]
        self.w_head = weights(s.d, s.vocab)
        self.prompt_qkv = [dense(*w) for w in self.w_qkv]
        self.prompt_out = [dense(*w) for w in self.w_out]
        self.norms = [(norm(), norm()) for _ in range(s.layers)]
        self.last_norm = norm()
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
        # what a slot was forked from: a number for the fork, and the tokens that its slots share
        self.family = [(-1 - i, 0) for i in range(s.slots)]
        self.forks = 0

    def step(self, slots: list, tokens: list) -> list:
        """New tokens tokens[i] [n] of slot slots[i], all slots in one pass; returns their
        normed hidden states [n, d].  Slots of one fork stand next to one another."""
        s = self.s
        add = [0] * s.slots
        for i, x in zip(slots, tokens):
            add[i] += x.shape[0]
            self.held[i] += x.shape[0]
        moves, status = M.pages_reserve(self.refs, self.table, self.lens,
                                        torch.tensor(add, dtype=torch.int32, device="cuda"), s.page)
        if status.tolist() != [0, 0]:
            raise RuntimeError("the cache is full")
        M.pages_copy(self.cache, moves)
        new = [x.shape[0] for x in tokens]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
        rows = torch.tensor(slots, device="cuda")
        table, kv_len = self.table[rows], self.lens[rows]
        # runs of slots of one fork are the groups that share keys
        first = [n for n, i in enumerate(slots) if n == 0 or self.family[i][0] != self.family[slots[n - 1]][0]]
        groups, shared = i32(first + [len(slots)]), i32([self.family[slots[n]][1] for n in first])
        ends = first[1:] + [len(slots)]
        hints = dict(max_q=max(new), max_group=max(sum(new[a:b]) for a, b in zip(first, ends)),
                     max_shared=max(self.family[i][1] for i in slots),
                     max_tail=max(self.held[i] - self.family[i][1] for i in slots))
        # the stream, and what is added to it next: every norm does that
        x = self.embedding[torch.cat(tokens).long()]
        more = torch.zeros_like(x)
        # Beyond 16 tokens linear4 reads the weights more than once; without a fork's slots
        # next to one another there are no keys to read together.
        prompt, lone = x.shape[0] > 16, len(first) == len(slots)
        for l in range(s.layers):
            if prompt:
                y, x = M.rms_norm(more, self.norms[l][0], residual=x)
                qkv = y @ self.prompt_qkv[l].T
            else:
                y, scale, x = M.rms_norm(more, self.norms[l][0], residual=x, out_dtype=torch.int8, group=64)
                qkv = M.linear4(y, *self.w_qkv[l], x_scale=scale)
            q, k, v = qkv.view(-1, s.hq + 2 * s.hk, s.dim).split([s.hq, s.hk, s.hk], 1)
            kp, vp = self.cache[2 * l], self.cache[2 * l + 1]
            q = M.rope_append(q, k, v, kp, vp, table, cu, kv_len, self.freq, mscale=self.mscale)
            if lone:
                o = M.paged_attention(q, kp, vp, table, cu, kv_len, max_q=max(new),
                                      max_kv=max(self.held[i] for i in slots))
            else:
                o = M.paged_attention_shared(q, kp, vp, table, cu, kv_len, groups, shared, **hints)
            o = o.view(-1, s.hq * s.dim)
            o = o @ self.prompt_out[l].T if prompt else M.linear4(o, *self.w_out[l])
            y, x = M.rms_norm(o, self.norms[l][1], residual=x)
            more = self.moe[l].forward(y)
        y, _ = M.rms_norm(more, self.last_norm, residual=x)
        return list(y.split(new))

    def choose(self, hidden: torch.Tensor) -> torch.Tensor:
        """The next token of every row of hidden states [B, d]."""
        logits = M.linear4(hidden, *self.w_head, out_dtype=torch.float32)
        u = torch.rand(hidden.shape[0], device="cuda", generator=self.g)
        return M.sample(logits, u, temperature=0.8, top_k=50, top_p=0.95)

    def fork(self, src: int, dst: list):
        i32 = dict(dtype=torch.int32, device="cuda")
        M.pages_fork(self.refs, self.table, self.lens, torch.full((len(dst),), src, **i32),
                     torch.tensor(dst, **i32))
        self.forks += 1
        for i in [src] + dst:
            self.held[i] = self.held[src]
            self.family[i] = (self.forks, self.held[src])

    def release(self, slots: list):
        M.pages_free(self.refs, self.table, self.lens,
                     torch.tensor(slots, dtype=torch.int32, device="cuda"))
        for i in slots:
            self.held[i] = 0
            self.family[i] = (-1 - i, 0)
        moves, count = M.pages_compact(self.refs, self.table)
        M.pages_copy(self.cache, moves, count)

    def pages_in_use(self) -> int:
        return int((self.refs > 0).sum())


def run(seed: int = 0):
    """The loop; returns (relative error of the decoded continuation against the
    same tokens read as one prompt, pages in use before and after compaction)."""
    s = Shape()
    srv = Server(s, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    prompt = torch.randint(0, s.vocab, (75,), dtype=torch.int32, device="cuda", generator=g)
    for a, b in ((0, 40), (40, 75)):                  # the prompt, in chunks
        hidden = srv.step([0], [prompt[a:b]])[0]
    srv.fork(0, [1, 2, 3])
    live, texts = [1, 2, 3], {i: [] for i in (1, 2, 3)}

    def decode(hidden, steps):
        for _ in range(steps):
            tokens = srv.choose(hidden)
            for n, i in enumerate(live):
                texts[i].append(tokens[n:n + 1])
            hidden = torch.cat(srv.step(live, [texts[i][-1] for i in live]))
        return hidden

    hidden = decode(hidden[-1:].expand(3, -1).contiguous(), 4)   # three continuations, token by token
    before = srv.pages_in_use()
    srv.release([0, 2])
    after = srv.pages_in_use()
    live, hidden = [1, 3], hidden[[0, 2]]
    hidden = decode(hidden, 4)
    live, hidden = [3, 1], hidden[[1, 0]]
    last = decode(hidden, 1)[:1]
    whole = srv.step([5], [torch.cat([prompt] + texts[3])])[0][-1:]
    err = ((last.float() - whole.float()).norm() / whole.float().norm()).item()
    if M.paged_device_error():
        raise RuntimeError("device error")
    return err, before, after


if __name__ == "__main__":
    e, before, after = run()
    print(f"continuation against one prompt: relative error {e:.2e}; "
          f"pages in use {before} -> {after}")
