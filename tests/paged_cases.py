"""Seeded inputs and error bounds shared by the paged-cache tests."""
import numpy as np
import torch

from oracle import paged_oracle as PO


def u_of(dtype):
    """Largest relative error of one rounding to dtype: half a step."""
    return torch.finfo(dtype).eps / 2


def values(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make_batch(seed, new, kv, page, hk, d, dtype, hq, extra=3, device="cpu", width=None, fill=None):
    """A batch of sequences in scattered pages.  ``fill``: what the cache holds
    where no sequence has a token (default: random numbers like the rest)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-x // page) for x in kv]
    P = sum(need) + extra
    width = width or max(max(need, default=0) + 1, 1)
    perm = torch.randperm(P, generator=g)
    table = torch.full((len(kv), width), -1, dtype=torch.int32)
    k = torch.randn(P, page, hk, d, generator=g).to(dtype)
    v = torch.randn(P, page, hk, d, generator=g).to(dtype)
    held = torch.zeros(P, page, dtype=torch.bool)
    at = 0
    for n, (c, x) in enumerate(zip(need, kv)):
        table[n, :c] = perm[at:at + c].to(torch.int32)
        for i in range(c):
            held[perm[at + i], :max(0, min(page, x - i * page))] = True
        at += c
    if fill is not None:
        k[~held] = fill
        v[~held] = fill
    q = (2 * torch.randn(sum(new), hq, d, generator=g)).to(dtype)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    kv_len = torch.tensor(kv, dtype=torch.int32)
    b = dict(q=q, k=k, v=v, table=table, cu=cu, kv_len=kv_len)
    return {n: t.to(device) for n, t in b.items()}


def attention_reference(b, scale, causal=True, window=0):
    return PO.attention(values(b["q"]), np.nan_to_num(values(b["k"]), posinf=0, neginf=0),
                        np.nan_to_num(values(b["v"]), posinf=0, neginf=0),
                        b["table"].cpu().numpy(), b["cu"].cpu().numpy(), b["kv_len"].cpu().numpy(),
                        scale, causal, window)


def attention_bars(ref, dtype, d, kv):
    """Allowed error of o and lse, per element.

    A score is a sum of d exact products in fp32, times the scale: off by at
    most (d + 4) 2^-24 z, with z its sum of magnitudes, and its weight by that
    much relatively; an exponential by 2^-21; a sum of kv terms by kv 2^-24.
    The weights are rounded once to dtype (u) and so is the result (u)."""
    o, lse, a, z = ref
    u = u_of(dtype)
    f = ((d + 4) * z + kv + 64) * 2.0 ** -24 + 2.0 ** -21
    bar_o = u * (1 + u) * a + u * np.abs(o) + 2 * f[..., None] * a + 1e-30
    bar_l = f + 4 * 2.0 ** -24 * np.abs(np.where(np.isfinite(lse), lse, 0))
    if dtype is torch.float16:  # subnormal weights and results: an absolute step
        bar_o = bar_o + 2.0 ** -24 * (1 + kv * 4.0)
    return bar_o, bar_l


def check_attention(o, lse, ref, dtype, d, kv):
    o_ref, l_ref = ref[0], ref[1]
    bo, bl = attention_bars(ref, dtype, d, kv)
    o = values(o)
    inside = ~np.isnan(o_ref)
    assert np.all(np.abs(o - o_ref)[inside] <= bo[inside]), (
        f"o off by {np.max((np.abs(o - o_ref) / bo)[inside]):.3f} of the bar")
    if lse is not None:
        x = values(lse)
        rows = ~np.isnan(l_ref)
        empty = rows & np.isneginf(l_ref)
        assert np.all(np.isneginf(x[empty])), "lse of a row that sees nothing"
        fine = rows & np.isfinite(l_ref)
        assert np.all(np.abs(x - l_ref)[fine] <= bl[fine]), (
            f"lse off by {np.max((np.abs(x - l_ref) / bl)[fine]):.3f} of the bar")


def page_state(seed, S, width, P, page, share=True):
    """A consistent state: slots of random lengths, some sharing their first pages."""
    rng = np.random.default_rng(seed)
    perm = rng.permutation(P)
    refs = np.zeros(P, np.int32)
    table = np.full((S, width), -1, np.int32)
    lens = np.zeros(S, np.int32)
    at = 0
    for s in range(S):
        if rng.random() < 0.2:
            continue
        n = int(rng.integers(1, max(width * page // 2, 1) + 1))
        c = -(-n // page)
        first = 0
        if share and s and lens[s - 1] and rng.random() < 0.5:
            first = int(min(c, -(-int(lens[s - 1]) // page)))
            if first == c and n % page and rng.random() < 0.5:
                n = min(n, int(lens[s - 1]))
                c = first = -(-n // page)
            table[s, :first] = table[s - 1, :first]
        if at + c - first > P:
            table[s] = -1
            continue
        table[s, first:c] = perm[at:at + c - first]
        at += c - first
        lens[s] = n
        for p in table[s, :c]:
            refs[p] += 1
    return refs, table, lens
