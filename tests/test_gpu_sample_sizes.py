"""sample over many rows of vocabularies of all sizes, on either side of those at which a row
takes more blocks or a block takes an SM alone: the same tokens as in a batch of a few rows,
which the definition decides."""
import pytest
import torch

import sparse_moe_bit_gb300 as M
from tests.test_gpu_sample import BF, FP, logits, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [8192, 16393, 16394, 32793, 32794, 40001, 49152, 65593, 65594, 70000, 98305, 131193, 131194,
                               151936, 200001])
def test_many_rows_as_in_small_batches(V):
    base, u4 = logits(V, 4, V, FP if V % 2 else BF)
    z = base.cuda().repeat(80, 1)
    u = torch.rand(320, device="cuda", generator=torch.Generator(device="cuda").manual_seed(V))
    u[:4] = u4.cuda()
    for kw in (dict(top_p=0.9), dict(top_k=50, top_p=0.95), dict(top_k=3000), dict(temperature=0.0), dict(min_p=0.01)):
        tok, lp = M.sample(z, u, **kw, return_logprobs=True)
        for at in (0, 8, 152, 312):
            t8, l8 = M.sample(z[at:at + 8], u[at:at + 8], **kw, return_logprobs=True)
            assert torch.equal(t8, tok[at:at + 8]) and torch.equal(l8, lp[at:at + 8])
        names = dict(top_p="p", top_k="k", temperature="t", min_p="m")
        few = run(base, u4, **{names[n]: v for n, v in kw.items()})
        assert few.tolist() == tok[:4].tolist()
