"""paged_attention_shared where some sequences bring chunks of a prompt beside others that
decode: every token finds its sequence and its group."""
import pytest
import torch

import sparse_moe_bit_gb300 as M
from tests.test_gpu_paged_shared import batch, check, hints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,prefix,tail,outside", [
    ([1], [0], 5, (0, 0)), ([3, 2], [40, 17], 30, (1, 1)), ([40], [90], 3, (0, 2)), ([2, 1, 35], [64, 0, 20], 9, (33, 0))],
    ids=str)
@pytest.mark.parametrize("nq", [8, 9, (0, 40), (1, 150)], ids=str)
@pytest.mark.parametrize("hint", [False, True])
def test_chunks_beside_single_tokens(groups, prefix, tail, outside, nq, hint):
    b, new, kv = batch(13, groups, prefix, tail, nq, 16, 1, 64, torch.bfloat16, 2, outside=outside)
    check(b, kv, **(hints(b, new, kv) if hint else {}))


def test_a_long_chunk():
    """Thousands of new tokens of one sequence between continuations of another prompt."""
    b, new, kv = batch(14, [3, 1, 3], [50, 0, 33], 20, 1, 16, 2, 64, torch.bfloat16, 4)
    n = 4099
    pages = -(-n // 16)
    P = b["k"].shape[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in ("k", "v"):
        b[x] = torch.cat([b[x], torch.randn(pages, 16, 2, 64, device="cuda", generator=g).to(b[x].dtype)])
    table = torch.full((7, pages), -1, dtype=torch.int32, device="cuda")
    w = b["table"].shape[1]
    table[:, :w] = b["table"]
    table[3] = torch.arange(P, P + pages)
    b["table"] = table
    kv[3] = n
    new[3] = n
    i32 = dict(dtype=torch.int32, device="cuda")
    b["kv_len"] = torch.tensor(kv, **i32)
    b["cu"] = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), **i32)
    b["q"] = torch.randn(sum(new), 4, 64, device="cuda", generator=g).to(b["q"].dtype)
    o, lse = M.paged_attention_shared(*(b[x] for x in ("q", "k", "v", "table", "cu", "kv_len", "cu_group", "shared")),
                                      return_lse=True)
    args = [b[x] for x in ("q", "k", "v", "table", "cu", "kv_len")]
    plain, plain_lse = M.paged_attention(*args, return_lse=True)
    args[2] = args[2].abs()
    most = M.paged_attention(*args).double()       # the weights' sum of magnitudes
    torch.cuda.synchronize()
    assert M.paged_device_error() == 0
    # Either side rounds weights and result by half a step of bf16 (and `most` is off by as
    # much); scores are sums of 64 products and the sums have 4099 terms, in fp32.
    z = b["q"].double().norm(dim=-1).max() * max(b["k"].double().norm(dim=-1).max(), 1) / 8
    f = ((64 + 4) * z + n + 64) * 2.0 ** -24 + 2.0 ** -21
    u = 2.0 ** -8
    assert ((lse - plain_lse).abs() <= 2 * f + 8 * 2.0 ** -24 * plain_lse.abs()).all()
    bar = 2 * (u * (1 + u) * most * (1 + 2 * u) + u * plain.double().abs() * (1 + u) + 2 * f * most) + 1e-30
    assert ((o.double() - plain.double()).abs() <= bar).all()
