"""paged_attention_shared against the fp64 definition of attention over the cache."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from tests.paged_cases import attention_reference, check_attention, make_batch

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def batch(seed, groups, prefix, tail, nq, page, hk, d, dtype, hq, fill=None, outside=(0, 0)):
    """Groups of sequences whose first prefix[g] keys are the same: whole pages shared, what is
    left of a page copied; ``outside``: lone sequences before and behind the groups."""
    rng = np.random.default_rng(seed)
    sizes = [1] * outside[0] + list(groups) + [1] * outside[1]
    shared = [0] * outside[0] + list(prefix) + [0] * outside[1]
    new, kv = [], []
    for m, p in zip(sizes, shared):
        for _ in range(m):
            n = nq if isinstance(nq, int) else int(rng.integers(nq[0], nq[1] + 1))
            new.append(n)
            kv.append(p + n + int(rng.integers(0, tail + 1)))
    b = make_batch(seed, new, kv, page, hk, d, dtype, hq, fill=fill)
    at = 0
    for m, p in zip(sizes, shared):
        whole, part = p // page, p % page
        for i in range(at + 1, at + m):
            b["table"][i, :whole] = b["table"][at, :whole]
            if part:
                a, c = int(b["table"][at, whole]), int(b["table"][i, whole])
                for x in ("k", "v"):
                    b[x][c, :part] = b[x][a, :part]
        at += m
    b = {n: t.cuda() for n, t in b.items()}
    first = outside[0]
    b["cu_group"] = torch.tensor(np.cumsum([first] + list(groups)), dtype=torch.int32, device="cuda")
    b["shared"] = torch.tensor(list(prefix), dtype=torch.int32, device="cuda")
    return b, new, kv


ARGS = ("q", "k", "v", "table", "cu", "kv_len", "cu_group", "shared")


def attend(b, **kw):
    return M.paged_attention_shared(*(b[x] for x in ARGS), return_lse=True, **kw)


def check(b, kv, causal=True, **kw):
    d = b["q"].shape[2]
    o, lse = attend(b, causal=causal, **kw)
    torch.cuda.synchronize()
    assert M.paged_device_error() == 0
    ref = attention_reference(b, d ** -0.5, causal)
    check_attention(o, lse, ref, b["q"].dtype, d, max(kv))
    return o, lse


def hints(b, new, kv):
    g = b["cu_group"].tolist()
    s = b["shared"].tolist()
    per = [0] * len(kv)
    for i, p in enumerate(s):
        for n in range(g[i], g[i + 1]):
            per[n] = p
    return dict(max_q=max(new), max_group=max(sum(new[g[i]:g[i + 1]]) for i in range(len(s))),
                max_shared=max(s), max_tail=max(k - p for k, p in zip(kv, per)))


@pytest.mark.parametrize("groups,prefix,tail,nq", [
    ([2], [1], 0, 1), ([2], [40], 5, 1), ([4], [150], 30, 1), ([3, 2], [64, 65], 70, 1), ([1], [90], 9, 1),
    ([5, 1, 3], [100, 50, 31], 20, 2), ([2, 2], [0, 17], 40, 1), ([9], [300], 0, 1), ([20], [257], 3, 3),
    ([3], [10], 200, 17), ([40], [513], 33, 1), ([2, 30], [400, 100], 5, 5)], ids=str)
@pytest.mark.parametrize("dim,hk,group", [(64, 2, 4), (128, 1, 8), (256, 2, 8), (128, 3, 1)])
@pytest.mark.parametrize("hint", [False, True])
def test_groups(groups, prefix, tail, nq, dim, hk, group, hint):
    b, new, kv = batch(7, groups, prefix, tail, nq, 16, hk, dim, BF, hk * group)
    check(b, kv, **(hints(b, new, kv) if hint else {}))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 48, 100, 256])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_pages_and_types(page, dtype):
    for groups, prefix in (([4], [201]), ([30, 2], [130, 77])):
        b, new, kv = batch(page, groups, prefix, 60, 1, page, 2, 128, dtype, 8, fill=float("nan"), outside=(1, 2))
        check(b, kv, **hints(b, new, kv))


@pytest.mark.parametrize("members,prefix,tail", [(3, 5000, 10), (48, 3000, 300), (64, 130, 900), (2, 9, 4000)])
@pytest.mark.parametrize("nq", [1, (0, 4)], ids=str)
def test_longer_contexts(members, prefix, tail, nq):
    b, new, kv = batch(members, [members], [prefix], tail, nq, 64, 2, 256, BF, 16, fill=float("nan"))
    check(b, kv, **hints(b, new, kv))


def test_not_causal():
    b, new, kv = batch(3, [3, 4], [50, 60], 30, 4, 16, 2, 64, BF, 8)
    check(b, kv, causal=False, **hints(b, new, kv))


def test_shared_lengths_that_do_not_fit():
    """What a sequence has before its new tokens bounds the shared keys; a negative length is 0."""
    b, new, kv = batch(4, [3, 3, 2], [80, 33, 20], 12, 3, 16, 2, 64, BF, 8)
    want, _ = check(b, kv)
    room = [min(kv[n] - new[n] for n in range(a, z)) for a, z in ((0, 3), (3, 6), (6, 8))]
    # (the members agree on no more than the prefix: lengths above it only where one of them ends there)
    kv2 = list(kv)
    for i in range(2):
        kv2[3 * i] = [80, 33][i] + new[3 * i]
    b["kv_len"].copy_(torch.tensor(kv2, dtype=torch.int32))
    for s in ([10 ** 9, 2 ** 31 - 1, 20], [81, 34, -5], [-2 ** 31, 33, 20]):
        b["shared"].copy_(torch.tensor(s, dtype=torch.int32))
        check(b, kv2)
    assert min(room) > 0 and want.isfinite().all()


def test_sequences_without_new_tokens():
    """Finished members, the first of a group among them, whose rows hold no pages."""
    b, new, kv = batch(5, [3, 2, 4], [70, 40, 90], 20, 2, 16, 2, 128, BF, 8)
    new2, cu = list(new), [0]
    for n in (0, 4, 6, 7):
        new2[n] = 0
    for n in new2:
        cu.append(cu[-1] + n)
    keep = torch.cat([torch.arange(2 * n, 2 * n + 2) for n in range(9) if new2[n]]).cuda()
    b["q"] = b["q"][keep].contiguous()
    b["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for n in (0, 4):
        b["table"][n] = -1
        b["kv_len"][n] = 0
    check(b, [k if new2[n] else 0 for n, k in enumerate(kv)])


def test_contexts_shorter_than_their_new_tokens():
    """Tokens before position 0 see nothing, and their group then shares nothing."""
    b, new, kv = batch(6, [3], [30], 10, 4, 16, 2, 64, BF, 8)
    b["kv_len"][1] = 2
    o, lse = check(b, kv)
    assert (o[4:6] == 0).all() and lse[4:6].isneginf().all()
    b["kv_len"][1] = 0
    o, lse = check(b, kv)
    assert (o[4:8] == 0).all() and lse[4:8].isneginf().all()


def test_bad_groups_and_pages_stay_inside():
    b, new, kv = batch(8, [3, 3], [64, 32], 20, 1, 16, 2, 64, BF, 8)
    plain, _ = M.paged_attention(*(b[x] for x in ARGS[:6]), return_lse=True)
    for cu in ([-5, 3, 6], [0, 6, 3], [7, 9, 11], [0, 0, 0], [6, 3, 0], [-9, -8, 100]):
        b["cu_group"].copy_(torch.tensor(cu, dtype=torch.int32))
        b["shared"].fill_(0 if cu in ([0, 6, 3], [-9, -8, 100], [6, 3, 0]) else 16)
        o, _ = attend(b)
        torch.cuda.synchronize()
        assert torch.allclose(o.float(), plain.float(), atol=0.02, rtol=0.02), cu
    assert M.paged_device_error() == 0
    # a bad page among the shared ones is left out for all of the group
    b["cu_group"].copy_(torch.tensor([0, 3, 6], dtype=torch.int32))
    b["shared"].copy_(torch.tensor([64, 32], dtype=torch.int32))
    b["table"][:3, 1] = 10 ** 6
    o, lse = attend(b)
    torch.cuda.synchronize()
    assert M.paged_device_error() == M.PAGED_DEVERR_PAGE
    k2 = {n: t.clone() for n, t in b.items()}
    d = 64
    ref = attention_reference({**k2, "table": torch.where(k2["table"] == 10 ** 6, -1, k2["table"])}, d ** -0.5)
    check_attention(o, lse, ref, BF, d, max(kv))
    for cu_q in ([0, 6, 2, 9, 1, 3, 6], [-3, 50, 2, 2, 2, 2, 1]):
        b["cu"].copy_(torch.tensor(cu_q, dtype=torch.int32))
        attend(b)
    b["kv_len"].copy_(torch.tensor([2 ** 31 - 1, -7, 0, 3, 10 ** 8, 1], dtype=torch.int32))
    attend(b)
    torch.cuda.synchronize()
    M.paged_device_error()


def test_no_groups_no_tokens():
    b, new, kv = batch(9, [2, 2], [20, 20], 9, 1, 16, 2, 64, BF, 8)
    o, lse = M.paged_attention(*(b[x] for x in ARGS[:6]), return_lse=True)
    b["cu_group"], b["shared"] = b["cu_group"][:1].contiguous(), b["shared"][:0]
    o2, lse2 = attend(b)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    b["q"] = b["q"][:0]
    assert attend(b)[0].shape == (0, 8, 64)


def test_rows_outside_every_sequence_stay():
    b, new, kv = batch(10, [3], [40], 9, 1, 16, 2, 64, BF, 8)
    q = torch.cat([b["q"], b["q"]])
    out = torch.full((6, 3, 8, 64), 3.0, dtype=BF, device="cuda")[:, 1]
    want, _ = check(b, kv)
    b["q"] = q
    o, _ = attend(b, out=out)
    assert o is out and torch.equal(out[:3], want) and (out[3:] == 3).all()


def test_streams_graphs_and_repeats():
    b, new, kv = batch(11, [12, 1, 5], [900, 30, 333], 150, 1, 64, 2, 128, BF, 16)
    h = hints(b, new, kv)
    want = check(b, kv, **h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [attend(b, stream=side, **h) for _ in range(6)]
    here = [attend(b, **h) for _ in range(6)]
    torch.cuda.current_stream().wait_stream(side)
    for x in got + here:
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(b["q"])
    with torch.cuda.graph(graph):
        attend(b, out=out, **h)
    graph.replay()
    assert torch.equal(out, want[0])
    # the same graph over lengths that have changed on the GPU
    b["kv_len"].sub_(1)
    b["shared"].sub_(1)
    graph.replay()
    assert torch.equal(out, check(b, [k - 1 for k in kv], **h)[0])


def test_workspace_of_the_caller():
    import ctypes

    from sparse_moe_bit_gb300 import paged
    b, new, kv = batch(12, [4], [200], 20, 1, 16, 2, 128, BF, 8)
    want, _ = check(b, kv)
    n = ctypes.c_size_t()
    lib = paged._library()
    assert lib.paged_attention_shared_workspace(paged._cache(b["k"], b["v"]),
                                                paged._batch(b["table"], b["cu"], b["kv_len"], 4), 8, 1, 0, 0, 0,
                                                0, ctypes.byref(n)) == 0
    ws = torch.full((n.value + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    o, _ = attend(b, workspace=ws[:n.value])
    assert torch.equal(o, want) and (ws[n.value:] == 0xAB).all()
    with pytest.raises(M.MoEError, match="workspace"):
        attend(b, workspace=ws[:n.value - 1])


@pytest.mark.parametrize("dim", [64, 256])
def test_a_workspace_at_any_sixteen_bytes(dim):
    """Parts are written a sector at once where the workspace lies on one, in halves elsewhere."""
    b, new, kv = batch(23, [40], [3000], 30, 4, 16, 2, dim, BF, 16)
    plain = [b[x] for x in ("q", "k", "v", "table", "cu", "kv_len")]
    first = attend(b, **hints(b, new, kv))[0], M.paged_attention(*plain)
    ws = torch.zeros((64 << 20) + 64, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 32 == 0
    for at in (0, 16, 32, 48):
        o, _ = attend(b, workspace=ws[at:], **hints(b, new, kv))
        assert torch.equal(o, first[0])
        assert torch.equal(M.paged_attention(*plain, workspace=ws[at:]), first[1])
    torch.cuda.synchronize()
    assert M.paged_device_error() == 0
    check(b, kv, workspace=ws[16:], **hints(b, new, kv))


def test_next_to_fork_and_reserve():
    """The serving path: a prompt is forked, pages reserved and copied on write, new keys
    appended, and the continuations attend together."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(BF)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    freq, mscale = M.rope_frequencies(32, device="cuda")
    pools = torch.zeros(2, 40, 16, 2, 64, dtype=BF, device="cuda")
    refs, lens = torch.zeros(40, dtype=torch.int32, device="cuda"), i32(0, 0, 0, 0)
    table = torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
    for new in ([70, 0, 0, 0], [1, 1, 1, 1], [1, 1, 1, 1]):
        if new[1] and int(lens[1]) == 0:
            M.pages_fork(refs, table, lens, i32(0, 0, 0), i32(1, 2, 3))
        moves, status = M.pages_reserve(refs, table, lens, i32(*new), 16)
        M.pages_copy(pools, moves)
        T = sum(new)
        cu = torch.cat([i32(0), i32(*new).cumsum(0).to(torch.int32)])
        q = M.rope_append(rand(T, 8, 64), rand(T, 2, 64), rand(T, 2, 64), pools[0], pools[1], table, cu, lens, freq)
        assert status.tolist() == [0, 0]
        b = dict(q=q, k=pools[0], v=pools[1], table=table, cu=cu, kv_len=lens, cu_group=i32(0, 4), shared=i32(70))
        check(b, lens.tolist())
