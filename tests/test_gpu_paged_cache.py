"""Rotary positions, the cache's append and the page operations
(include/paged.h) against their definitions in oracle/paged_oracle.py.

Rotation bound, per feature with pair (a, b): the angle in half turns is a
float (off by 2^-25) of the top 32 bits of the turn (2^-31), sin and cos are
off by 2^-23, mscale and the two products and the sum round once each at 2^-24;
|error| <= 10 * 2^-24 (|a| + |b|) mscale, and one rounding to the type."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from oracle import paged_oracle as PO
from tests.paged_cases import make_batch, page_state, u_of, values

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def _near(y, ref, bound, dtype):
    bar = 10 * 2.0 ** -24 * bound + u_of(dtype) * np.abs(ref) * (1 + 1e-3)
    if dtype is FP:
        bar = bar + 2.0 ** -25   # half a subnormal step
    err = np.abs(values(y) - ref)
    assert np.all(err <= bar), f"off by {np.max(err / np.maximum(bar, 1e-300)):.3f} of the bar"


def _freq(r, base=10000.0):
    return torch.tensor([base ** (-i / r) for i in range(r)], dtype=torch.float64)


@pytest.mark.parametrize("inverse", [False, True], ids=["forward", "gradient"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,D,r", [(1, 1, 2, 1), (7, 3, 64, 32), (33, 5, 80, 25), (5, 2, 256, 32),
                                     (2000, 2, 128, 64), (3, 1, 130, 8), (1, 4, 1024, 512)])
def test_rope(T, H, D, r, dtype, inter, inverse):
    g = torch.Generator().manual_seed(T + D)
    x = torch.randn(T, H, D, generator=g).to(dtype)
    pos = torch.randint(-10, 1 << 20, (T,), generator=g, dtype=torch.int32)
    f = _freq(r)
    y = M.rope(x.cuda(), pos.cuda(), f.cuda(), mscale=1.21, interleaved=inter, inverse=inverse)
    ref = PO.rope(values(x), pos.numpy(), f.numpy(), np.float32(1.21), inter, inverse)
    bound = PO.rope_bound(values(x), f.numpy(), 1.21, inter)
    _near(y, ref, bound, dtype)
    if 2 * r < D:   # the rest of the head passes bit for bit
        assert torch.equal(y.cpu()[..., 2 * r:], x[..., 2 * r:])


@pytest.mark.parametrize("inter", [False, True])
def test_rope_far_positions_and_custom_frequencies(inter):
    """Positions to 2^31, frequencies above a radian and negative ones."""
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32)
    f = torch.tensor([1.0, 3.7, -0.3, 1e-9, 100.25, 2e-5, 0.0, 6.283185307179586], dtype=torch.float64)
    x = torch.randn(6, 2, 16, generator=torch.Generator().manual_seed(3))
    y = M.rope(x.cuda(), pos.cuda(), f.cuda(), interleaved=inter)
    # the reference's own angle: exact product of integers of the doubles, modulo a turn
    from fractions import Fraction
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    ang = np.zeros((6, 8))
    for i, p in enumerate(pos.tolist()):
        for j, w in enumerate(f.tolist()):
            a = Fraction(w) * p
            ang[i, j] = float(a - (a // two_pi) * two_pi)
    ref = values(x).copy()
    ia = np.arange(0, 16, 2) if inter else np.arange(8)
    ib = ia + (1 if inter else 8)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = ref[..., ia].copy(), ref[..., ib].copy()
    ref[..., ia], ref[..., ib] = a * c - b * s, a * s + b * c
    bound = PO.rope_bound(values(x), f.numpy(), 1.0, inter)
    # the fp64 product f / (2 pi) rounds at 2^-53 twice: pos * turns * 2^-52 of a turn
    extra = np.abs(pos.numpy().astype(np.float64))[:, None] * np.abs(f.numpy()) * 2.0 ** -52
    e = np.zeros_like(ref)
    e[..., ia] = extra[:, None] * bound[..., ia]
    e[..., ib] = extra[:, None] * bound[..., ib]
    err = np.abs(values(y) - ref)
    assert np.all(err <= 10 * 2.0 ** -24 * bound + 2.0 ** -24 * np.abs(ref) + e)


def test_rope_views_and_in_place():
    """A misaligned view (the scalar path), a strided output, and in place."""
    f = _freq(16).cuda()
    base = torch.randn(9, 5, 70, device="cuda").to(BF)
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 1000
    x = base[:, 1:4, 3:67]
    ref = PO.rope(values(x), pos.cpu().numpy(), f.cpu().numpy())
    bound = PO.rope_bound(values(x), f.cpu().numpy(), 1.0, False)
    buf = torch.full((9, 6, 64), 3.0, dtype=BF, device="cuda")
    _near(M.rope(x, pos, f, out=buf[:, 2:5]), ref, bound, BF)
    assert torch.all(buf[:, :2] == 3) and torch.all(buf[:, 5] == 3)
    y = M.rope(x, pos, f)
    z = base.clone()
    M.rope(z[:, 1:4, 3:67], pos, f, out=z[:, 1:4, 3:67])
    assert torch.equal(z[:, 1:4, 3:67], y)
    z[:, 1:4, 3:67] = base[:, 1:4, 3:67]
    assert torch.equal(z, base)


def test_rope_gradient_against_differences():
    """The inverse call is the gradient of the forward one: fp32 central
    differences of a random functional."""
    f = _freq(4).cuda()
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(3, 2, 12, device="cuda", generator=g)
    w = torch.randn(3, 2, 12, device="cuda", generator=g)
    pos = torch.tensor([0, 17, 4001], dtype=torch.int32, device="cuda")
    dx = M.rope(w, pos, f, mscale=0.9, inverse=True)
    h = 2.0 ** -3   # the map is linear: any step gives the derivative, a large one less noise
    for i in range(12):
        e = torch.zeros_like(x)
        e[..., i] = h
        up, dn = (M.rope(x + s * e, pos, f, mscale=0.9).double() for s in (1, -1))
        num = ((up - dn) * w.double()).sum(-1) / (2 * h)
        # features past the turning ones carry no mscale
        bar = 12 * 40 * 2.0 ** -24 * 8 / h
        assert torch.all((num - dx[..., i].double()).abs() <= bar)


@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("new,kv,page,d,hk,g,r", [
    ([1], [1], 16, 64, 1, 1, 32), ([1, 1, 1], [17, 300, 16], 16, 256, 2, 8, 32),
    ([5, 0, 40, 1], [5, 9, 100, 33], 24, 128, 3, 2, 64), ([2000, 3], [70000, 50], 64, 128, 1, 2, 60)])
def test_append(new, kv, page, d, hk, g, r, dtype, inter):
    b = make_batch(sum(kv), new, kv, page, hk, d, dtype, hk * g, device="cuda")
    T = sum(new)
    x = torch.randn(T, hk * (g + 2) + 1, d, device="cuda").to(dtype)   # q | k | v | unused
    q, k, v = x[:, :hk * g], x[:, hk * g:hk * (g + 1)], x[:, hk * (g + 1):hk * (g + 2)]
    f = _freq(r, 500000.0).cuda()
    kp, vp = b["k"].clone(), b["v"].clone()
    y = M.rope_append(q, k, v, kp, vp, b["table"], b["cu"], b["kv_len"], f, mscale=1.1, interleaved=inter)
    torch.cuda.synchronize()
    assert M.paged_device_error() == 0
    pos = np.concatenate([np.arange(c - n, c) for n, c in zip(new, kv)])
    seq = np.concatenate([np.full(n, i) for i, n in enumerate(new)])
    fn = f.cpu().numpy()
    m = np.float32(1.1)
    _near(y, PO.rope(values(q), pos, fn, m, inter), PO.rope_bound(values(q), fn, 1.1, inter), dtype)
    pg = b["table"].cpu().numpy()[seq, pos // page]
    idx = torch.from_numpy(pg).long().cuda(), torch.from_numpy(pos % page).cuda()
    _near(kp[idx], PO.rope(values(k), pos, fn, m, inter), PO.rope_bound(values(k), fn, 1.1, inter), dtype)
    assert torch.equal(vp[idx], v)
    # nothing else in the cache changed
    kp[idx], vp[idx] = b["k"][idx], b["v"][idx]
    assert torch.equal(kp, b["k"]) and torch.equal(vp, b["v"])


def test_append_leaves_out_what_has_no_place():
    """Tokens before position 0, with a bad page, outside every sequence."""
    b = make_batch(3, [4, 4, 4], [2, 40, 40], 16, 1, 64, BF, 2, device="cpu")
    b["table"][1, 2] = 99999            # positions 36.. of sequence 1: its whole chunk
    b["cu"] = torch.tensor([1, 4, 8, 10], dtype=torch.int32)   # tokens 0, 10, 11 belong to nobody
    b = {k: t.cuda() for k, t in b.items()}
    q, k, v = (torch.randn(12, h, 64, device="cuda").to(BF) for h in (2, 1, 1))
    f = _freq(8).cuda()
    kp, vp = b["k"].clone(), b["v"].clone()
    qo = torch.full_like(q, 9.0)
    M.rope_append(q, k, v, kp, vp, b["table"], b["cu"], b["kv_len"], f, q_out=qo)
    torch.cuda.synchronize()
    assert M.paged_device_error() == M.PAGED_DEVERR_PAGE
    for t in (0, 10, 11):
        assert torch.all(qo[t] == 9)
    pos = np.array([-1, 0, 1] + [36, 37, 38, 39] + [38, 39])   # kv 2 with 3 new tokens, and so on
    _near(qo[1:10], PO.rope(values(q[1:10]), pos, f.cpu().numpy()),
          PO.rope_bound(values(q[1:10]), f.cpu().numpy(), 1.0, False), BF)
    written = torch.zeros(b["k"].shape[:2], dtype=torch.bool, device="cuda")
    for n, p in ((0, 0), (0, 1), (2, 38), (2, 39)):
        written[b["table"][n, p // 16].long(), p % 16] = True
    assert torch.equal((vp != b["v"]).any(-1).any(-1), written)
    assert torch.equal((kp != b["k"]).any(-1).any(-1) & ~written, torch.zeros_like(written))


def test_append_in_place_and_head_major_cache():
    b = make_batch(4, [3, 1], [20, 40], 16, 2, 128, BF, 4, device="cuda")
    q, k, v = (torch.randn(4, h, 128, device="cuda").to(BF) for h in (4, 2, 2))
    f = _freq(64).cuda()
    k1, v1 = b["k"].clone(), b["v"].clone()
    want = M.rope_append(q, k, v, k1, v1, b["table"], b["cu"], b["kv_len"], f)
    k2, v2 = (b[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "kv")
    qi = q.clone()
    got = M.rope_append(qi, k, v, k2, v2, b["table"], b["cu"], b["kv_len"], f, q_out=qi)
    assert got.data_ptr() == qi.data_ptr() and torch.equal(got, want)
    assert torch.equal(k1, k2) and torch.equal(v1, v2)


# ---------------------------------------------------------------------- pages
def _dev(*a):
    return [torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in a]


def _same(dev, ref):
    for d, r in zip(dev, ref):
        assert np.array_equal(d.cpu().numpy(), r)


@pytest.mark.parametrize("S,W,P,page", [(1, 1, 1, 1), (7, 5, 40, 4), (60, 33, 1500, 16),
                                        (1500, 12, 9000, 8)])
def test_fork_reserve_free_compact(S, W, P, page):
    """The four operations in a row, each against its definition."""
    for seed in range(3):
        rng = np.random.default_rng(100 + seed)
        refs, table, lens = page_state(seed, S, W, P, page)
        r, t, l = _dev(refs, table, lens)
        # forks, some of them refused: full or repeated targets, numbers out of range, chains
        F = S + 3
        src, dst = rng.integers(-1, S + 1, F), rng.integers(-1, S + 1, F)
        refs, table, lens, refused = PO.fork(refs, table, lens, src, dst)
        n = torch.full((1,), 77, dtype=torch.int32, device="cuda")
        M.pages_fork(r, t, l, *_dev(src, dst), refused=n)
        _same((r, t, l), (refs, table, lens))
        assert n.item() == refused
        add = rng.integers(-2, 2 * page, S)
        add[(lens + add) > W * page] = 0
        refs, table, lens, moves, status = PO.reserve(refs, table, lens, add, page)
        m, st = M.pages_reserve(r, t, l, *_dev(add), page)
        _same((r, t, l, m, st), (refs, table, lens, moves, status))
        # what cannot be had changes nothing
        big = np.full(S, W * page + 1)
        *_, moves, status = PO.reserve(refs, table, lens, big, page)
        m, st = M.pages_reserve(r, t, l, *_dev(big), page)
        assert status[1] > 0
        _same((r, t, l, m, st), (refs, table, lens, moves, status))
        slots = rng.integers(-1, S + 1, S // 2 + 1)
        refs, table, lens = PO.free(refs, table, lens, slots)
        M.pages_free(r, t, l, *_dev(slots))
        _same((r, t, l), (refs, table, lens))
        refs, table, moves, count = PO.compact(refs, table)
        m, c = M.pages_compact(r, t)
        _same((r, t, m, c), (refs, table, moves, count))
        m, c = M.pages_compact(r, t)      # nothing is left to move
        assert c.item() == 0 and torch.all(m == -1)
        _same((r, t), (refs, table))


def test_reserve_when_pages_are_missing():
    refs, table, lens = page_state(3, 20, 10, 60, 4)
    r, t, l = _dev(refs, table, lens)
    add = np.where(10 * 4 - lens < 30, 10 * 4 - lens, 30)
    *_, moves, status = PO.reserve(refs, table, lens, add, 4)
    assert status[0] > 0 and status[1] == 0
    m, st = M.pages_reserve(r, t, l, *_dev(add), 4)
    _same((r, t, l, m, st), (refs, table, lens, moves, status))


def test_compact_of_all_free_all_used_and_stale_numbers():
    for refs in (np.zeros(10, int), np.ones(10, int), np.array([0] * 9 + [3]), np.array([1] + [0] * 4999 + [2])):
        # numbers of free pages and out of range in a table stay as they are
        table = np.array([[len(refs) - 1, -1, len(refs) + 5], [len(refs) - 2, 0, -7]])
        r, t = _dev(refs, table)
        a, b, moves, count = PO.compact(refs.astype(np.int32), table)
        m, c = M.pages_compact(r, t)
        _same((r, t, m, c), (a, b, moves, count))


def test_table_rows_apart():
    """A table that is a slice of a wider one: its neighbours stay."""
    refs, table, lens = page_state(5, 9, 6, 40, 4)
    wide = torch.full((9, 11), 123, dtype=torch.int32, device="cuda")
    wide[:, 2:8] = torch.from_numpy(table).cuda()
    r, l = _dev(refs, lens)
    add = np.minimum(3, 24 - lens)
    refs, table, lens, moves, status = PO.reserve(refs, table, lens, add, 4)
    M.pages_reserve(r, wide[:, 2:8], l, *_dev(add), 4)
    refs, table, lens = PO.free(refs, table, lens, [1, 4])
    M.pages_free(r, wide[:, 2:8], l, *_dev([1, 4]))
    refs, table, *_ = PO.compact(refs, table)
    M.pages_compact(r, wide[:, 2:8])
    _same((r, wide[:, 2:8], l), (refs, table, lens))
    assert torch.all(wide[:, :2] == 123) and torch.all(wide[:, 8:] == 123)


@pytest.mark.parametrize("shape,dtype", [((1, 5, 8), F32), ((3, 40, 16, 2, 64), BF), ((4, 9, 50000), FP),
                                         ((2, 30, 24), torch.uint8)])
def test_copy(shape, dtype):
    B, P = shape[:2]
    if dtype is torch.uint8:
        shape = (B, P, 48)
    base = torch.randint(0, 100, (B, P + 2) + shape[2:], device="cuda").to(dtype)
    pools = base[:, 1:P + 1]                # arrays further apart than their pages
    perm = np.random.default_rng(P).permutation(P)
    moves = np.full((P, 2), -1)
    k = P // 2
    moves[:k, 0], moves[:k, 1] = perm[:k], perm[k:2 * k]
    moves[0, 1] = P                          # out of range, on both sides
    if k > 1:
        moves[1, 0] = -3
    moves = moves[np.random.default_rng(1).permutation(P)]
    want = base.clone()
    for a, b in moves:
        if 0 <= a < P and 0 <= b < P:
            want[:, 1 + b] = want[:, 1 + a]
    M.pages_copy(pools, *_dev(moves))
    assert torch.equal(base, want)


def test_copy_count():
    pools = torch.arange(8, device="cuda", dtype=torch.int32).reshape(1, 8, 1).repeat(2, 1, 4).contiguous()
    for count, want in ((0, 0), (1, 1), (2, 2), (99, 3), (-4, 0)):
        p = pools.clone()
        c, m = _dev(count, [[0, 4], [1, 5], [2, 6]])
        M.pages_copy(p, m, c)
        ref = pools.clone()
        for i in range(want):
            ref[:, 4 + i] = pools[:, i]
        assert torch.equal(p, ref)
