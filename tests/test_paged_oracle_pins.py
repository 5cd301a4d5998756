"""The fp64 definitions of the paged-cache operators against other things than
themselves: library routines, hand-worked states, invariants.  No GPU."""
import numpy as np
import pytest
import scipy.special as sp
import torch

from oracle import paged_oracle as PO
from tests.paged_cases import make_batch, page_state, values


def test_attention_is_softmax_over_a_dense_cache():
    b = make_batch(1, [3], [21], 8, 1, 64, torch.float32, 2)
    o, lse, _, _ = PO.attention(values(b["q"]), values(b["k"]), values(b["v"]), b["table"].numpy(),
                                b["cu"].numpy(), b["kv_len"].numpy(), 0.125)
    ids = b["table"][0, :3].long()
    K, V = values(b["k"][ids]).reshape(-1, 64)[:21], values(b["v"][ids]).reshape(-1, 64)[:21]
    for i in range(3):
        z = 0.125 * values(b["q"])[i] @ K[:19 + i].T
        np.testing.assert_allclose(o[i], sp.softmax(z, -1) @ V[:19 + i], rtol=1e-12)
        np.testing.assert_allclose(lse[i], sp.logsumexp(z, -1), rtol=1e-12)


def test_window_and_empty_rows():
    b = make_batch(2, [4], [2], 4, 1, 64, torch.float32, 1)   # two tokens before position 0
    o, lse, _, _ = PO.attention(values(b["q"]), values(b["k"]), values(b["v"]), b["table"].numpy(),
                                b["cu"].numpy(), b["kv_len"].numpy(), 1.0, window=1)
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:2]))
    # a window of one sees the token itself
    page = values(b["v"][b["table"][0, 0].item()])
    np.testing.assert_allclose(o[2:, 0], page[:2, 0], rtol=1e-12)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_is_a_rotation(inter):
    rng = np.random.default_rng(0)
    x, f = rng.standard_normal((5, 2, 20)), np.array([1.0, 0.25, 0.01])
    pos = np.array([0, 1, 5, 1000, -3])
    y = PO.rope(x, pos, f, 1.0, inter)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 6:], x[..., 6:])
    ia = [0, 2, 4] if inter else [0, 1, 2]
    ib = [1, 3, 5] if inter else [3, 4, 5]
    z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * pos[:, None, None] * f)
    np.testing.assert_allclose(y[..., ia] + 1j * y[..., ib], z, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(PO.rope(y, pos, f, 1.0, inter, inverse=True), x, atol=1e-12)
    # scores depend on the difference of positions alone
    s0 = (PO.rope(x[:1], [7], f, 1.0, inter) * PO.rope(x[1:2], [4], f, 1.0, inter)).sum(-1)
    s1 = (PO.rope(x[:1], [107], f, 1.0, inter) * PO.rope(x[1:2], [104], f, 1.0, inter)).sum(-1)
    np.testing.assert_allclose(s0, s1, rtol=1e-10)


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_rope_is_the_gradient(inter):
    rng = np.random.default_rng(1)
    x, dy, f, m = rng.standard_normal((2, 1, 8)), rng.standard_normal((2, 1, 8)), np.array([1.0, .1]), 1.3
    dx = PO.rope(dy, [3, 9], f, m, inter, inverse=True)
    num = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        num[i] = ((PO.rope(x + e, [3, 9], f, m, inter) - PO.rope(x - e, [3, 9], f, m, inter)) * dy).sum() / 2e-6
    # (features that do not turn pass their gradient unchanged)
    np.testing.assert_allclose(dx, num, atol=1e-8)


def _counts(refs, table, lens, page):
    c = np.zeros(len(refs), int)
    for s in range(len(lens)):
        used = table[s][table[s] >= 0]
        assert len(used) == -(-lens[s] // page) and np.all(table[s][:len(used)] >= 0)
        np.add.at(c, used, 1)
    return c


@pytest.mark.parametrize("seed", range(8))
def test_page_operations_keep_the_state_consistent(seed):
    page, S, W, P = 4, 12, 9, 80
    refs, table, lens = page_state(seed, S, W, P, page)
    assert np.array_equal(_counts(refs, table, lens, page), refs)
    empty, full = np.where(lens == 0)[0], np.where(lens > 0)[0]
    refs, table, lens, refused = PO.fork(refs, table, lens, np.resize(full, len(empty)), empty)
    assert refused == 0 and np.array_equal(_counts(refs, table, lens, page), refs)
    add = np.random.default_rng(seed).integers(0, 6, S)
    before, held = lens.copy(), table.copy()
    refs, table, lens, moves, status = PO.reserve(refs, table, lens, add, page)
    assert status == (0, 0) and np.array_equal(lens, before + add)
    assert np.array_equal(_counts(refs, table, lens, page), refs)
    for s in range(S):
        if add[s] and before[s] % page:      # the page that is written next is its own
            assert refs[table[s, before[s] // page]] == 1 or moves[s, 0] < 0
        if moves[s, 0] >= 0:
            assert held[s, before[s] // page] == moves[s, 0] and table[s, before[s] // page] == moves[s, 1]
    refs, table, lens = PO.free(refs, table, lens, full[:3])
    assert np.array_equal(_counts(refs, table, lens, page), refs)
    content = {p: p * 10 for p in range(P)}
    seen = [[content[p] for p in row if p >= 0] for row in table]
    refs, table, moves, n = PO.compact(refs, table)
    for a, b in moves[:n]:
        content[b] = content[a]
    assert [[content[p] for p in row if p >= 0] for row in table] == seen
    live = int((refs > 0).sum())
    assert np.all(refs[:live] > 0) and np.all(refs[live:] == 0)


def test_hand_worked_reserve():
    # slot 0 holds 5 tokens in pages 2, 4 (page of 4), slot 1 shares both
    refs = np.array([0, 1, 2, 0, 2, 0])
    table = np.array([[2, 4, -1], [2, 4, -1], [1, -1, -1]])
    lens = np.array([5, 5, 4])
    r, t, l, moves, status = PO.reserve(refs, table, lens, np.array([1, 0, 1]), 4)
    assert status == (0, 0)
    assert t.tolist() == [[2, 0, -1], [2, 4, -1], [1, 3, -1]] and l.tolist() == [6, 5, 5]
    assert r.tolist() == [1, 1, 2, 1, 1, 0] and moves.tolist() == [[4, 0], [-1, -1], [-1, -1]]
    r, t, l, moves, status = PO.reserve(refs, table, lens, np.array([8, 8, 0]), 4)
    assert status == (0, 2) and np.array_equal(r, refs) and np.array_equal(l, lens)
    r, t, l, moves, status = PO.reserve(refs, table, lens, np.array([4, 4, 1]), 4)
    assert status == (2, 0) and np.array_equal(t, table)
