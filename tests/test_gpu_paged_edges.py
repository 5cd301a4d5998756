"""Narrow cases of the paged-cache calls (include/paged.h) on the GPU."""
import pytest
import torch

import sparse_moe_bit_gb300 as M
from tests.paged_cases import make_batch

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def test_host_tensors_are_refused():
    """One argument on the host: refused before anything is enqueued."""
    b = make_batch(1, [3], [20], 16, 2, 64, BF, 4, device="cuda")
    f = torch.ones(8, dtype=torch.float64)
    names = ("q", "k", "v", "table", "cu", "kv_len")
    for stream in (None, torch.cuda.Stream()):
        for n in names:
            a = dict(b, **{n: b[n].cpu()})
            with pytest.raises(ValueError):
                M.paged_attention(*(a[x] for x in names), stream=stream)
        with pytest.raises(ValueError):
            M.rope(b["q"], b["kv_len"].expand(3).contiguous(), f, stream=stream)
        with pytest.raises(ValueError):
            M.rope_append(b["q"], b["k"][:3, 0], b["v"][:3, 0], b["k"], b["v"], b["table"], b["cu"],
                          b["kv_len"], f, stream=stream)
        with pytest.raises(ValueError):
            M.pages_reserve(b["kv_len"], b["table"], b["kv_len"], torch.ones(1, dtype=torch.int32), 16,
                            stream=stream)
    torch.cuda.synchronize()
    assert M.paged_device_error() == 0
