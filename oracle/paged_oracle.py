"""Plain fp64 definitions of the paged-cache operators (test infrastructure
only; shares no code with the CUDA path and neither imports the other).

Arrays are numpy; 16-bit types come in as fp64 values.
"""
from __future__ import annotations

import numpy as np


# --------------------------------------------------------------------- rotary
def rope(x, pos, freq, mscale=1.0, interleaved=False, inverse=False):
    """x [T, H, D] fp64, pos [T], freq [r]: the first 2r features turn."""
    r = len(freq)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64)[None]
    c, s = np.cos(ang)[:, None] * mscale, np.sin(ang)[:, None] * mscale
    if inverse:
        s = -s
    y = np.array(x, np.float64)
    ia = np.arange(0, 2 * r, 2) if interleaved else np.arange(r)
    ib = ia + (1 if interleaved else r)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def rope_bound(x, freq, mscale, interleaved):
    """|a| + |b| of every feature's pair times mscale (0 where nothing turns)."""
    r = len(freq)
    y = np.zeros_like(x, np.float64)
    ia = np.arange(0, 2 * r, 2) if interleaved else np.arange(r)
    ib = ia + (1 if interleaved else r)
    m = (np.abs(x[..., ia]) + np.abs(x[..., ib])) * abs(mscale)
    y[..., ia] = m
    y[..., ib] = m
    return y


# ------------------------------------------------------------------ attention
def clamp_batch(cu, kv_len, T, capacity):
    """(first token, new tokens, context) of every sequence, as the ABI reads them."""
    out = []
    for n in range(len(kv_len)):
        t0 = min(max(int(cu[n]), 0), T)
        t1 = min(max(int(cu[n + 1]), t0), T)
        out.append((t0, t1 - t0, min(max(int(kv_len[n]), 0), capacity)))
    return out


def attention(q, k_pages, v_pages, table, cu, kv_len, scale, causal=True, window=0):
    """q [T, Hq, D], pages [P, page, Hk, D].  Returns o, lse, and for error
    bounds: a = sum_j p_j |v_j| (like o) and z = max_j scale sum_d |q_d k_jd|
    over visible keys (like lse).  Rows outside every sequence stay NaN."""
    T, Hq, D = q.shape
    P, page, Hk, _ = k_pages.shape
    o = np.full((T, Hq, D), np.nan)
    a = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    zb = np.full((T, Hq), np.nan)
    for n, (t0, nq, kv) in enumerate(clamp_batch(cu, kv_len, T, table.shape[1] * page)):
        j = np.arange(kv)
        pg = table[n][j // page] if kv else np.zeros(0, int)
        good = (pg >= 0) & (pg < P)
        K = np.zeros((kv, Hk, D))
        V = np.zeros((kv, Hk, D))
        K[good] = k_pages[pg[good], j[good] % page]
        V[good] = v_pages[pg[good], j[good] % page]
        for i in range(nq):
            pos = kv - nq + i
            see = good.copy()
            if causal or pos < 0:   # a token that stands before position 0 sees no key
                see &= j <= pos
            if window:
                see &= pos - j < window
            for h in range(Hq):
                g = h // (Hq // Hk)
                ks, vs = K[see, g], V[see, g]
                qi = q[t0 + i, h]
                if not len(ks):
                    o[t0 + i, h] = a[t0 + i, h] = 0.0
                    lse[t0 + i, h], zb[t0 + i, h] = -np.inf, 0.0
                    continue
                z = scale * (ks @ qi)
                m = z.max()
                p = np.exp(z - m)
                l = p.sum()
                o[t0 + i, h] = p @ vs / l
                a[t0 + i, h] = p @ np.abs(vs) / l
                lse[t0 + i, h] = m + np.log(l)
                zb[t0 + i, h] = scale * (np.abs(ks) @ np.abs(qi)).max()
    return o, lse, a, zb


# ---------------------------------------------------------------------- pages
def fork(refs, table, lens, src, dst):
    refs, table, lens = refs.copy(), table.copy(), lens.copy()
    old_t, old_l = table.copy(), lens.copy()
    S, refused = len(lens), 0
    for i, (s, d) in enumerate(zip(src, dst)):
        if (not 0 <= s < S or not 0 <= d < S or old_l[d] != 0 or d in list(dst[:i]) or s in list(dst)):
            refused += 1
            continue
        table[d], lens[d] = old_t[s], old_l[s]
        for pg in old_t[s]:
            if 0 <= pg < len(refs):
                refs[pg] += 1
    return refs, table, lens, refused


def reserve(refs, table, lens, add, page):
    S, width = table.shape
    refs, table, lens = refs.copy(), table.copy(), lens.copy()
    moves = np.full((S, 2), -1, np.int64)
    plan, narrow = [], 0
    for s in range(S):
        more = max(int(add[s]), 0)
        have, want = -(-int(lens[s]) // page), -(-(int(lens[s]) + more) // page)
        if more and want > width:
            narrow += 1
            want = have
        own = False
        if more and lens[s] % page and have <= width:
            last = table[s, have - 1]
            own = 0 <= last < len(refs) and refs[last] > 1
        plan.append((have, want, own))
    need = sum(w - h + int(o) for h, w, o in plan)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    status = (max(need - len(free), 0), narrow)
    if any(status):
        return refs, table, lens, moves, status
    give = iter(free)
    for s, (have, want, own) in enumerate(plan):
        if own:
            p = next(give)
            moves[s] = table[s, have - 1], p
            refs[table[s, have - 1]] -= 1
            refs[p] += 1
            table[s, have - 1] = p
        for c in range(have, want):
            p = next(give)
            refs[p] += 1
            table[s, c] = p
        lens[s] += max(int(add[s]), 0)
    return refs, table, lens, moves, status


def free(refs, table, lens, slots):
    refs, table, lens = refs.copy(), table.copy(), lens.copy()
    done = set()
    for s in slots:
        if 0 <= s < len(lens) and s not in done:
            done.add(s)
            for pg in table[s]:
                if 0 <= pg < len(refs):
                    refs[pg] -= 1
            table[s], lens[s] = -1, 0
    return refs, table, lens


def compact(refs, table):
    P = len(refs)
    live = int((refs > 0).sum())
    out = [p for p in range(P) if refs[p] > 0 and p >= live]
    hole = [p for p in range(P) if refs[p] <= 0 and p < live]
    refs, table = refs.copy(), table.copy()
    moves = np.full((P, 2), -1, np.int64)
    to = {}
    for i, (a, b) in enumerate(zip(out, hole)):
        moves[i] = a, b
        refs[b], refs[a] = refs[a], 0
        to[a] = b
    for e in np.ndindex(table.shape):
        table[e] = to.get(int(table[e]), table[e])
    return refs, table, moves, len(out)
