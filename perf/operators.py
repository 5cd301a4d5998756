"""Cases of the operators around the paged key/value cache: rotary positions
(alone, and fused with the write of new keys and values into the cache), the
attention of new tokens over the cache, and the cache's page maintenance.

Where ``own`` is false, ``run`` computes an operator in its plain form from
elementary torch operations; where it is true, through the framework's calls.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One user's next token: the smallest call of a serving loop, latency alone
        # (16 query heads on 2 key/value heads of 256, the attention layer's shape).
        dict(name="attend_decode_one", op="attend", dtype="bf16", n=1, nq=1, rest=1, kv=1027,
             hq=16, hk=2, d=256, page=16, window=0),
        # A decode batch of ragged contexts: every sequence's cache is read once.
        dict(name="attend_decode_batch", op="attend", dtype="bf16", n=64, nq=1, rest=1, kv=8192,
             hq=16, hk=2, d=256, page=64, window=0),
        # A mixed step: one prompt chunk next to sequences that verify a few drafted
        # tokens, three query heads to a key/value head, a sliding window.
        dict(name="attend_mixed_window", op="attend", dtype="fp16", n=9, nq=777, rest=3, kv=3001,
             hq=24, hk=8, d=128, page=48, window=1024),
        # A chunk of a long prompt over all of the prompt before it: compute alone.
        dict(name="attend_chunk_long", op="attend", dtype="bf16", n=1, nq=4096, rest=1, kv=32768,
             hq=16, hk=2, d=256, page=64, window=0),
        # A decode batch's new keys and values go into the cache; a quarter of the head turns.
        dict(name="append_decode", op="append", dtype="bf16", n=64, nq=1, rest=1, kv=8192, hq=16,
             hk=2, d=256, rot=64, page=64, layout="half", scaling="none"),
        # A prompt chunk far out in a long context, interleaved pairs, scaled frequencies.
        dict(name="append_chunk_far", op="append", dtype="fp16", n=3, nq=8191, rest=61, kv=200003,
             hq=32, hk=8, d=128, rot=128, page=32, layout="inter", scaling="yarn"),
        # Rotation alone, of one head group of a few tokens with an odd rotary size.
        dict(name="rope_small", op="rope", dtype="fp32", t=37, h=5, d=80, rot=50, kv=5000,
             layout="half", scaling="linear", inverse=False),
        # The gradient of a training batch's queries: the inverse rotation.
        dict(name="rope_gradient", op="rope", dtype="bf16", t=16385, h=32, d=128, rot=128,
             kv=16385, layout="half", scaling="banded", inverse=True),
        # One prompt forked into four continuations: the shared last page is copied on write.
        dict(name="fork_one", op="fork", dtype="bf16", n=1, each=4, kv=1500, seqs=8, pools=4,
             page=16, hk=2, d=256, add=1),
        # A beam step of a batch: many forks, every layer's pools.
        dict(name="fork_batch", op="fork", dtype="bf16", n=48, each=5, kv=4001, seqs=288,
             pools=20, page=64, hk=2, d=256, add=3),
        # A few finished sequences leave a small cache, and it is compacted.
        dict(name="compact_small", op="compact", dtype="fp16", pages=300, seqs=10, kv=400,
             pools=2, page=16, hk=8, d=64),
        # A long-running server's cache of ten layers gives half of itself back.
        dict(name="compact_large", op="compact", dtype="bf16", pages=4096, seqs=96, kv=4000,
             pools=20, page=64, hk=2, d=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "rope", "fork", "compact"])
    dt = rng.choice(["bf16", "fp16"])
    hk, d, g = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "attend":
        kind = rng.choice(["decode", "few", "mixed", "chunk"])
        kv = _log(rng, 40, 16384)
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        if kind == "decode":
            n, nq, rest = _log(rng, 1, 96), 1, 1
        elif kind == "few":
            n = _log(rng, 1, 32)
            nq = rest = rng.randint(2, 16)
        elif kind == "mixed":
            n, nq, rest, kv = rng.randint(2, 8), _log(rng, 17, 700), rng.randint(1, 5), _log(rng, 700, 4000)
        else:
            n, nq, rest = 1, _log(rng, 17, 2048), 1
        kv = max(min(kv, 160_000_000 // (n * hk * d)), 40)   # no more cache than the listed cases read
        nq, rest = min(nq, kv), min(rest, kv // 8 + 1)
        return dict(op="attend", dtype=dt, n=n, nq=nq, rest=rest, kv=kv, hq=hk * g, hk=hk, d=d,
                    page=page, window=window)
    if op == "append":
        n, nq = _log(rng, 1, 64), _log(rng, 1, 4096)
        kv = nq + min(_log(rng, 1, 100000), 160_000_000 // (n * hk * d))
        return dict(op="append", dtype=dt, n=n, nq=nq, rest=rng.randint(1, 9),
                    kv=kv, hq=hk * g, hk=hk, d=d,
                    rot=rng.choice([d, d // 2, d // 4]), page=page,
                    layout=rng.choice(["half", "inter"]),
                    scaling=rng.choice(["none", "linear", "yarn", "banded"]))
    if op == "rope":
        rot = 2 * rng.randint(4, d // 2)
        return dict(op="rope", dtype=rng.choice(["bf16", "fp16", "fp32"]), t=_log(rng, 1, 12000),
                    h=rng.randint(1, 32), d=d, rot=rot, kv=_log(rng, 12000, 1000000),
                    layout=rng.choice(["half", "inter"]),
                    scaling=rng.choice(["none", "linear", "yarn", "banded"]),
                    inverse=rng.random() < 0.5)
    if op == "fork":
        n, each = _log(rng, 1, 48), rng.randint(1, 5)
        return dict(op="fork", dtype=dt, n=n, each=each, kv=_log(rng, 20, 4000),
                    seqs=n * (1 + each) + rng.randint(0, 20), pools=2 * rng.randint(1, 6),
                    page=page, hk=hk, d=64, add=rng.randint(1, 150))
    seqs = rng.randint(2, 64)
    kv = _log(rng, 30, 2000)
    return dict(op="compact", dtype=dt, pages=seqs * -(-kv // page) + rng.randint(0, 300),
                seqs=seqs, kv=kv, pools=2 * rng.randint(1, 6), page=page, hk=hk, d=64)


# ------------------------------------------------------------- what a case is
def _new(c):
    """New tokens of each sequence."""
    return [c["nq"]] + [c["rest"]] * (c["n"] - 1)


def _lens(c):
    """Context of each sequence, new tokens included: ragged from an eighth of the
    longest to the longest, the first the longest."""
    n, kv = c["n"], c["kv"]
    return [max(q, kv - (i * 7919 % n) * (kv - kv // 8) // n) for i, q in enumerate(_new(c))]


def _frequencies(c, dev="cpu"):
    """Radians a position of every rotary pair in 64 bits, and the factor on cos and sin."""
    rot, base = c["rot"], 10000.0 if c["scaling"] == "none" else 500000.0
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if c["scaling"] == "linear":
        return (f / 4.0).to(dev), 1.0
    if c["scaling"] == "yarn":  # factor 8 over 32768 positions, 32 and 1 turns
        lo, hi = ((rot * math.log(32768 / (t * 2 * math.pi)) / (2 * math.log(base))) for t in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return (f / 8.0 * ramp + f * (1 - ramp)).to(dev), 0.1 * math.log(8.0) + 1.0
    if c["scaling"] == "banded":  # factor 8 over 8192 positions, bands at 1 and 4 turns
        turns = 8192 * f / (2 * math.pi)
        s = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (f * (s + (1 - s) / 8.0)).to(dev), 1.0
    return f.to(dev), 1.0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, dt, *shape):
    out = torch.empty(shape, dtype=dt, device="cuda")
    return out.normal_(generator=g)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(lens, page, width, total, g):
    """A table of pages scattered over the cache: the pages of each sequence in order, -1 behind them."""
    need = torch.tensor([-(-x // page) for x in lens])
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width)[None]
    at = (need.cumsum(0) - need)[:, None] + col
    held = col < need[:, None]
    return torch.where(held.cuda(), perm[torch.where(held, at, 0).cuda()], -1).contiguous()


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = _DT[c["dtype"]]
    s = dict(case=c)
    if c["op"] in ("attend", "append"):
        lens, new = _lens(c), _new(c)
        width = -(-max(lens) // c["page"]) + 1
        total = sum(-(-x // c["page"]) for x in lens) + 3
        s["table"] = _tables(lens, c["page"], width, total, g)
        s["cu"] = _i32([0] + torch.tensor(new).cumsum(0).tolist())
        s["kv_len"] = _i32(lens)
        s["max_q"], s["max_kv"] = max(new), max(lens)
        t = sum(new)
        pool = _randn(g, dt, 2, total, c["page"], c["hk"], c["d"])
        s["k"], s["v"] = pool[0], pool[1]
        if c["op"] == "attend":
            # queries that give peaked scores; what lies behind a sequence's end in its last
            # page is whatever was there, not numbers
            s["q"] = _randn(g, dt, t, c["hq"], c["d"]).mul_(2.0)
            last = s["table"].gather(1, ((s["kv_len"] - 1) // c["page"]).long()[:, None])[:, 0].long()
            behind = torch.arange(c["page"], device="cuda")[None] > ((s["kv_len"] - 1) % c["page"])[:, None]
            bad = torch.zeros(total, c["page"], dtype=torch.bool, device="cuda")
            bad[last] = behind
            pool.masked_fill_(bad[None, :, :, None, None], float("nan"))
            s["scale"] = c["d"] ** -0.5
        else:
            # the projection's output: queries, keys and values of a token side by side
            h = c["hq"] + 2 * c["hk"]
            x = _randn(g, dt, t, h, c["d"])
            s["q"], s["new_k"], s["new_v"] = x.split([c["hq"], c["hk"], c["hk"]], 1)
            f, s["mscale"] = _frequencies(c)
            s["freq"] = f.cuda()
        return s
    if c["op"] == "rope":
        x = _randn(g, dt, c["t"], c["h"] + 1, c["d"])
        s["x"] = x[:, 1:]
        # packed documents: positions that start over, up to the longest context
        s["pos"] = (torch.arange(c["t"], device="cuda") * 7 % c["kv"]).to(torch.int32)
        f, s["mscale"] = _frequencies(c)
        s["freq"] = f.cuda()
        return s
    per = c["page"] * c["hk"] * c["d"]
    if c["op"] == "fork":
        n, need = c["n"], -(-c["kv"] // c["page"])
        lens = [c["kv"] - i * (c["kv"] // 3) // n for i in range(n)]
        extra = n * c["each"] * (-(-(c["add"]) // c["page"]) + 2)
        total = n * need + extra + 5
        width = -(-(c["kv"] + c["add"]) // c["page"]) + 2
        rows = _tables(lens, c["page"], width, total, g)
        s["table"] = torch.full((c["seqs"], width), -1, dtype=torch.int32, device="cuda")
        s["table"][:n] = rows
        s["lens"] = _i32(lens + [0] * (c["seqs"] - n))
        s["refs"] = torch.zeros(total, dtype=torch.int32, device="cuda")
        s["refs"][rows[rows >= 0].long()] = 1
        pair = torch.arange(n * c["each"], device="cuda", dtype=torch.int32)
        s["src"], s["dst"] = pair // c["each"], pair + n
        s["add"] = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda")
        s["add"][n:n + n * c["each"]] = c["add"]
    else:
        # sequences in pages scattered over the cache, every fourth one sharing the first
        # half of its pages with the one before; half of them are finished
        lens = [c["kv"] - i * (c["kv"] // 2) // c["seqs"] for i in range(c["seqs"])]
        width = -(-c["kv"] // c["page"]) + 1
        total = c["pages"]
        total = max(total, sum(-(-x // c["page"]) for x in lens))
        t = _tables(lens, c["page"], width, total, g)
        half = torch.arange(width, device="cuda") < ((_i32(lens) // c["page"]) // 2)[:, None]
        share = half & (torch.arange(c["seqs"], device="cuda") % 4 == 3)[:, None]
        s["table"] = torch.where(share, t.roll(1, 0), t).contiguous()
        s["lens"] = _i32(lens)
        held = torch.where(s["table"] >= 0, s["table"], total).long()
        s["refs"] = torch.zeros(total + 1, dtype=torch.int32, device="cuda").scatter_add_(
            0, held.reshape(-1), torch.ones(held.numel(), dtype=torch.int32, device="cuda"))[:total].clone()
        s["done"] = torch.randperm(c["seqs"], generator=g, device="cuda")[:c["seqs"] // 2].to(torch.int32)
    s["pools"] = _randn(g, dt, c["pools"], s["refs"].numel(), per)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_attend(s):
    c = s["case"]
    q, table, cu, kvl = s["q"], s["table"].long(), s["cu"].long(), s["kv_len"].long()
    dev, hk, g = q.device, c["hk"], c["hq"] // c["hk"]
    j = torch.arange(s["max_kv"], device=dev)
    i = torch.arange(s["max_q"], device=dev)
    held = j[None] < kvl[:, None]
    at = torch.where(held, table[:, j // c["page"]], 0)
    zero = torch.zeros((), device=dev)
    k = torch.where(held[..., None, None], s["k"][at, j % c["page"]].float(), zero)
    v = torch.where(held[..., None, None], s["v"][at, j % c["page"]].float(), zero)
    new = cu[1:] - cu[:-1]
    tok = (cu[:-1, None] + i[None]).clamp(max=q.shape[0] - 1)
    x = q[tok].float().reshape(c["n"], len(i), hk, g, c["d"])
    score = torch.matmul(x.permute(0, 2, 1, 3, 4).reshape(c["n"], hk, len(i) * g, c["d"]),
                         k.permute(0, 2, 3, 1)) * s["scale"]
    pos = (kvl - new)[:, None] + i[None]
    see = held[:, None] & (j[None, None] <= pos[..., None])
    if c["window"]:
        see &= j[None, None] > pos[..., None] - c["window"]
    see = see[:, None, :, None].expand(-1, 1, -1, g, -1).reshape(c["n"], 1, len(i) * g, len(j))
    score.masked_fill_(~see, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, zero)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    lse = (total.log() + top)[..., 0]
    o = o.reshape(c["n"], hk, len(i), g, c["d"]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.reshape(c["n"], hk, len(i), g).permute(0, 2, 1, 3).flatten(2, 3)
    t = torch.arange(q.shape[0], device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return o[seq, t - cu[seq]].to(q.dtype), lse[seq, t - cu[seq]]


def _rotate(x, pos, freq, mscale, layout, sign):
    """The rotation of the first pairs of every head: angles in 64 bits, products in 32."""
    r = freq.numel()
    angle = pos.double()[:, None] * freq[None]
    cos = (angle.cos() * mscale).float()[:, None]
    sin = (angle.sin() * (mscale * sign)).float()[:, None]
    y = x.float()
    if layout == "half":
        a, b, rest = y[..., :r], y[..., r:2 * r], y[..., 2 * r:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1).to(x.dtype)
    a, b, rest = y[..., 0:2 * r:2], y[..., 1:2 * r:2], y[..., 2 * r:]
    both = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([both, rest], -1).to(x.dtype)


def _plain_append(s):
    c = s["case"]
    cu, kvl = s["cu"].long(), s["kv_len"].long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = kvl[seq] - cu[seq + 1] + t
    page = s["table"].long()[seq, pos // c["page"]]
    s["k"][page, pos % c["page"]] = _rotate(s["new_k"], pos, s["freq"], s["mscale"], c["layout"], 1.0)
    s["v"][page, pos % c["page"]] = s["new_v"]
    return _rotate(s["q"], pos, s["freq"], s["mscale"], c["layout"], 1.0), s["k"], s["v"]


def _plain_copy(pools, moves):
    m = moves[moves[:, 0] >= 0].long()
    pools[:, m[:, 1]] = pools[:, m[:, 0]]


def _plain_fork(s):
    c = s["case"]
    refs, table, lens = s["refs"].clone(), s["table"].clone(), s["lens"].clone()
    page = c["page"]
    # fork: the new sequences hold the same pages
    src, dst = s["src"].long(), s["dst"].long()
    rows = table[src]
    table[dst], lens[dst] = rows, lens[src]
    pages = torch.where(rows >= 0, rows, refs.numel()).long().reshape(-1)
    refs = torch.cat([refs, refs.new_zeros(1)]).index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))[:-1]
    # reserve: a shared last page that is not full is exchanged for one of its own, then new ones
    have, want = (lens + page - 1) // page, (lens + s["add"] + page - 1) // page
    last = table.gather(1, (have - 1).clamp(min=0).long()[:, None])[:, 0]
    partly = (s["add"] > 0) & (lens % page > 0)
    own_copy = partly & (refs[last.clamp(min=0).long()] > 1)
    need = (want - have) + own_copy.int()
    first = need.cumsum(0) - need
    free = torch.argsort((refs != 0).int(), stable=True).to(torch.int32)
    col = torch.arange(table.shape[1], device=table.device)[None]
    begin = have - own_copy.int()
    new = (col >= begin[:, None]) & (col < want[:, None])
    rank = first[:, None] + col - begin[:, None]
    given = free[torch.where(new, rank, 0).long()]
    old = torch.where(own_copy, last, -1)
    moves = torch.stack([old, torch.where(own_copy, free[torch.where(own_copy, first, 0).long()], -1)], 1)
    table = torch.where(new, given, table)
    gone = torch.where(own_copy, last, refs.numel()).long()
    more = torch.where(new, given, refs.numel()).long().reshape(-1)
    refs = torch.cat([refs, refs.new_zeros(1)])
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    refs.index_add_(0, more, torch.ones_like(more, dtype=torch.int32))
    refs, lens = refs[:-1].contiguous(), lens + s["add"]
    _plain_copy(s["pools"], moves)
    return refs, table, lens, moves.to(torch.int32), s["pools"]


def _plain_compact(s):
    refs, table, lens = s["refs"].clone(), s["table"].clone(), s["lens"].clone()
    done, p = s["done"].long(), refs.numel()
    rows = table[done]
    pages = torch.where(rows >= 0, rows, p).long().reshape(-1)
    refs = torch.cat([refs, refs.new_zeros(1)]).index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))[:-1]
    table[done], lens[done] = -1, 0
    live, ids = refs > 0, torch.arange(p, device=refs.device)
    count = live.sum()
    out, hole = live & (ids >= count), ~live & (ids < count)
    src = torch.argsort((~out).int(), stable=True)
    dst = torch.argsort((~hole).int(), stable=True)
    used = ids < out.sum()
    moves = torch.stack([torch.where(used, src, -1), torch.where(used, dst, -1)], 1).to(torch.int32)
    rank = out.long().cumsum(0) - 1
    to = torch.where(out, dst[rank.clamp(min=0)], ids).to(torch.int32)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], table)
    refs = torch.where(hole, refs[src[(hole.long().cumsum(0) - 1).clamp(min=0)]], torch.where(out, 0, refs))
    _plain_copy(s["pools"], moves)
    return refs.to(torch.int32), table, lens, moves, out.sum().to(torch.int32), s["pools"]


# ----------------------------------------------------------------------- run
def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "attend":
            return _plain_attend(s)
        if c["op"] == "append":
            return _plain_append(s)
        if c["op"] == "rope":
            return _rotate(s["x"], s["pos"], s["freq"], s["mscale"], c["layout"], -1.0 if c["inverse"] else 1.0)
        return _plain_fork(s) if c["op"] == "fork" else _plain_compact(s)
    import sparse_moe_bit_gb300 as M
    if c["op"] == "attend":
        return M.paged_attention(s["q"], s["k"], s["v"], s["table"], s["cu"], s["kv_len"],
                                 scale=s["scale"], window=c["window"], max_q=s["max_q"],
                                 max_kv=s["max_kv"], return_lse=True)
    if c["op"] == "append":
        q = M.rope_append(s["q"], s["new_k"], s["new_v"], s["k"], s["v"], s["table"], s["cu"],
                          s["kv_len"], s["freq"], mscale=s["mscale"],
                          interleaved=c["layout"] == "inter")
        return q, s["k"], s["v"]
    if c["op"] == "rope":
        return M.rope(s["x"], s["pos"], s["freq"], mscale=s["mscale"],
                      interleaved=c["layout"] == "inter", inverse=c["inverse"])
    refs, table, lens = s["refs"].clone(), s["table"].clone(), s["lens"].clone()
    if c["op"] == "fork":
        M.pages_fork(refs, table, lens, s["src"], s["dst"])
        moves = M.pages_reserve(refs, table, lens, s["add"], c["page"])[0]
        M.pages_copy(s["pools"], moves)
        return refs, table, lens, moves, s["pools"]
    M.pages_free(refs, table, lens, s["done"])
    moves, count = M.pages_compact(refs, table)
    M.pages_copy(s["pools"], moves, count)
    return refs, table, lens, moves, count, s["pools"]


# ---------------------------------------------------------------------- work
def _seen(c):
    """Per sequence: (query, key) pairs that are visible, and keys that some query sees."""
    pairs = keys = 0
    for q, kv in zip(_new(c), _lens(c)):
        w = c["window"] or kv
        lo = max(0, kv - q - w + 1)
        keys += kv - lo
        first = kv - q + 1                      # keys that the first query sees, by causality
        grow = max(0, min(q, w - first + 1))    # queries that see fewer than w + 1 keys
        pairs += grow * first + grow * (grow - 1) // 2 + (q - grow) * w
    return pairs, keys


def work(case):
    c, e = case, _SIZE[case["dtype"]]
    if c["op"] == "attend":
        pairs, keys = _seen(c)
        t = sum(_new(c))
        return dict(bytes=2 * e * keys * c["hk"] * c["d"] + 2 * e * t * c["hq"] * c["d"] + 4 * t * c["hq"],
                    flops=4 * pairs * c["hq"] * c["d"])
    if c["op"] == "append":
        t = sum(_new(c))
        return dict(bytes=2 * e * t * (c["hq"] + 2 * c["hk"]) * c["d"],
                    flops=3 * t * (c["hq"] + c["hk"]) * c["rot"])
    if c["op"] == "rope":
        n = c["t"] * c["h"]
        return dict(bytes=2 * e * n * c["d"] + 4 * c["t"], flops=3 * n * c["rot"])
    per = c["page"] * c["hk"] * c["d"] * e * c["pools"]
    if c["op"] == "fork":
        lens = [c["kv"] - i * (c["kv"] // 3) // c["n"] for i in range(c["n"])]
        copies = c["each"] * sum(x % c["page"] > 0 for x in lens)
        width = -(-(c["kv"] + c["add"]) // c["page"]) + 2
        return dict(bytes=2 * per * copies + 8 * c["seqs"] * width, flops=0)
    lens = [c["kv"] - i * (c["kv"] // 2) // c["seqs"] for i in range(c["seqs"])]
    total = max(c["pages"], sum(-(-x // c["page"]) for x in lens))
    live = sum(-(-x // c["page"]) for x in lens) // 2
    moved = live * (total - live) // total     # what of a random half lies above its own number
    width = -(-c["kv"] // c["page"]) + 1
    return dict(bytes=2 * per * moved + 8 * c["seqs"] * width + 8 * total, flops=0)


# --------------------------------------------------------------------- exact
def exact(case, seed):
    """The definition, sequence by sequence and in 64 bits."""
    c, s = case, prepare(case, seed)
    if c["op"] == "attend":
        if 4.0 * sum(a * b for a, b in zip(_new(c), _lens(c))) * c["hq"] * c["d"] > 6e12:
            return None
        outs, lses = [], []
        at = 0
        for n, (nq, kv) in enumerate(zip(_new(c), _lens(c))):
            ids = s["table"][n].long()
            rows = -(-kv // c["page"])
            k = s["k"][ids[:rows]].flatten(0, 1)[:kv].double()
            v = s["v"][ids[:rows]].flatten(0, 1)[:kv].double()
            q = s["q"][at:at + nq].double()
            at += nq
            where = torch.arange(kv - nq, kv, device="cuda")[:, None]
            key = torch.arange(kv, device="cuda")[None]
            hide = key > where
            if c["window"]:
                hide |= where - key >= c["window"]
            o, l = [], []
            for h in range(c["hq"]):
                kh = h // (c["hq"] // c["hk"])
                z = (q[:, h] @ k[:, kh].T) * s["scale"]
                z = z.masked_fill(hide, -math.inf)
                lh = torch.logsumexp(z, 1)
                o.append(torch.exp(z - lh[:, None]) @ v[:, kh])
                l.append(lh)
            outs.append(torch.stack(o, 1))
            lses.append(torch.stack(l, 1))
        return torch.cat(outs), torch.cat(lses)

    def turn(x, pos, sign):
        f, m = _frequencies(c, "cuda")
        z = m * torch.exp(1j * sign * pos.double()[:, None] * f)
        y = x.double().clone()
        r = f.numel()
        if c["layout"] == "half":
            w = torch.complex(y[..., :r].contiguous(), y[..., r:2 * r].contiguous()) * z[:, None]
            y[..., :r], y[..., r:2 * r] = w.real, w.imag
        else:
            w = torch.complex(y[..., 0:2 * r:2].contiguous(), y[..., 1:2 * r:2].contiguous()) * z[:, None]
            y[..., 0:2 * r:2], y[..., 1:2 * r:2] = w.real, w.imag
        return y

    if c["op"] == "rope":
        return turn(s["x"], s["pos"], -1 if c["inverse"] else 1)
    if c["op"] == "append":
        pos = torch.cat([torch.arange(kv - nq, kv, device="cuda") for nq, kv in zip(_new(c), _lens(c))])
        k, v = s["k"], s["v"]
        k, v = k.double(), v.double()
        nk = turn(s["new_k"], pos, 1)
        at = 0
        for n, (nq, kv) in enumerate(zip(_new(c), _lens(c))):
            p = pos[at:at + nq]
            page = s["table"][n].long()[p // c["page"]]
            k[page, p % c["page"]] = nk[at:at + nq]
            v[page, p % c["page"]] = s["new_v"][at:at + nq].double()
            at += nq
        return turn(s["q"], pos, 1), k, v
    return None
