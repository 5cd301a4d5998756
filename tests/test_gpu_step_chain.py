"""A decode step of forked continuations as it is used, operator behind operator: norm
with the residual, projections, rotary positions and the cache, attention over the shared
prompt, projection, norm, logits, sampling, each against the definition on the same inputs;
and the whole chain captured in a graph."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from oracle import step_oracle as SO
from tests.paged_cases import attention_reference, check_attention
from tests.step_cases import linear4_bar, values, weights4

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
D, HQ, HK, DIM, VOCAB, PAGE = 512, 8, 2, 64, 3001, 16


class Step:
    def __init__(self, members, prompt, seed=0):
        g = torch.Generator().manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.n = members
        self.w = {k: [t.cuda() for t in weights4(seed + i, o, kk, 64, HF)] for i, (k, o, kk) in
                  enumerate((("qkv", (HQ + 2 * HK) * DIM, D), ("out", D, HQ * DIM), ("head", VOCAB, D)))}
        self.norm = [(1 + 0.2 * torch.randn(D, generator=g)).to(BF).cuda() for _ in range(2)]
        self.freq, _ = M.rope_frequencies(DIM, device="cuda")
        self.pools = torch.randn(2, 64, PAGE, HK, DIM, generator=g).to(BF).cuda()
        self.refs, self.lens = torch.zeros(64, **i32), torch.zeros(members, **i32)
        self.table = torch.full((members, 12), -1, **i32)
        add = torch.zeros(members, **i32)
        add[0] = prompt
        M.pages_reserve(self.refs, self.table, self.lens, add, PAGE)
        others = torch.arange(1, members, **i32)
        M.pages_fork(self.refs, self.table, self.lens, torch.zeros_like(others), others)
        moves, status = M.pages_reserve(self.refs, self.table, self.lens, torch.ones(members, **i32), PAGE)
        M.pages_copy(self.pools, moves)
        assert status.tolist() == [0, 0]
        self.cu = torch.arange(members + 1, **i32)
        self.groups, self.shared = torch.tensor([0, members], **i32), torch.tensor([prompt], **i32)
        self.x = torch.randn(members, D, generator=g).to(BF).cuda()
        self.r = torch.randn(members, D, generator=g).to(BF).cuda()
        self.u = torch.rand(members, generator=g).cuda()

    def run(self):
        t = {}
        t["y8"], t["s8"], t["h"] = M.rms_norm(self.x, self.norm[0], residual=self.r, out_dtype=torch.float8_e4m3fn,
                                              group=128)
        t["qkv"] = M.linear4(t["y8"], *self.w["qkv"], x_scale=t["s8"])
        q, k, v = t["qkv"].view(-1, HQ + 2 * HK, DIM).split([HQ, HK, HK], 1)
        t["q"] = M.rope_append(q, k, v, self.pools[0], self.pools[1], self.table, self.cu, self.lens, self.freq)
        t["o"], t["lse"] = M.paged_attention_shared(t["q"], self.pools[0], self.pools[1], self.table, self.cu,
                                                    self.lens, self.groups, self.shared, return_lse=True)
        t["out"] = M.linear4(t["o"].view(self.n, HQ * DIM), *self.w["out"])
        t["z"], t["h2"] = M.rms_norm(t["out"], self.norm[1], residual=t["h"])
        t["logits"] = M.linear4(t["z"], *self.w["head"], out_dtype=FP)
        t["token"], t["logprob"] = M.sample(t["logits"], self.u, 0.7, 40, 0.9, return_logprobs=True)
        return t


def _linear(x, w, y, dtype, bf16):
    ref = SO.linear4(x, w[0].cpu().numpy(), values(w[1]), values(w[2]))
    bar = linear4_bar(x, w[0].cpu().numpy(), values(w[1]), values(w[2]), ref, dtype, bf16)
    assert np.all(np.abs(values(y) - ref) <= bar)


@pytest.mark.parametrize("members,prompt", [(2, 5), (4, 100), (20, 33)])
def test_chain(members, prompt):
    s = Step(members, prompt)
    t = s.run()
    torch.cuda.synchronize()
    assert M.paged_device_error() == 0
    n, h = SO.rms_norm(values(s.x), values(s.norm[0]), values(s.r))
    y8 = t["y8"].float().double().cpu().numpy() * np.repeat(values(t["s8"]), 128, 1)
    top = np.repeat(np.abs(n.reshape(members, -1, 128)).max(-1), 128, 1)
    assert np.all(np.abs(y8 - n) <= np.maximum(np.abs(n) * 2.0 ** -4, top * 2.0 ** -10 / 448) * 1.001 + 1e-4 * np.abs(n))
    _linear(y8, s.w["qkv"], t["qkv"], BF, False)
    kv = s.lens.tolist()
    b = dict(q=t["q"], k=s.pools[0], v=s.pools[1], table=s.table, cu=s.cu, kv_len=s.lens)
    check_attention(t["o"], t["lse"], attention_reference(b, DIM ** -0.5), BF, DIM, max(kv))
    _linear(values(t["o"].view(members, -1)), s.w["out"], t["out"], BF, True)
    n2, h2 = SO.rms_norm(values(t["out"]), values(s.norm[1]), values(t["h"]))
    assert np.all(np.abs(values(t["z"]) - n2) <= (2.0 ** -8 + D * 2.0 ** -24) * np.abs(n2) + 1e-30)
    assert np.all(np.abs(values(t["h2"]) - h2) <= 2.0 ** -8 * np.abs(h2) * 1.001 + 1e-30)
    _linear(values(t["z"]), s.w["head"], t["logits"], FP, True)
    for i in range(members):
        ref = {SO.sample(values(t["logits"][i]), float(s.u[i]) + e, float(np.float32(0.7)), 40,
                         float(np.float32(0.9)) * (1 + f)) for e in (-2.0 ** -32, 0, 2.0 ** -32)
               for f in (-2.0 ** -32, 0, 2.0 ** -32)}
        assert int(t["token"][i]) in {r[0] for r in ref}
        assert min(abs(float(t["logprob"][i]) - r[1]) for r in ref) < 1e-5


def test_chain_in_a_graph_and_on_two_streams():
    s = Step(6, 70)
    want = s.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.run()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k].float(), want[k].float()) for k in want)
    # another batch's chain on another stream at the same time
    o, side = Step(9, 41, seed=50), torch.cuda.Stream()
    alone = o.run()
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = [o.run() for _ in range(4)]
    here = [s.run() for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(x[k].float(), alone[k].float()) for x in there for k in alone)
    assert all(torch.equal(x[k].float(), want[k].float()) for x in here for k in want)
    assert M.paged_device_error() == 0
