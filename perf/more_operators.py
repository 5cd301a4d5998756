"""Cases of the operators that a decode step of forked continuations has next to the MoE
block and the paged cache: the residual's addition with the RMS norm, products with 4-bit
weights, attention over a prompt that several sequences share, and the next token's choice.

Where ``own`` is false, ``run`` computes an operator in its plain form from elementary
torch operations; where it is true, through the framework's calls.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
       "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "int8": 1}
_TOP = {"e4m3": 448.0, "int8": 127.0}
_EPS = 1e-6


# --------------------------------------------------------------------- cases
def listed():
    return [
        # The residual stream of one user's next token, before a projection: latency alone.
        dict(name="norm_decode_one", op="norm", dtype="bf16", t=1, h=1, d=2048, gap=0, add=True,
             out="bf16", group=0, unit=False),
        # A prompt's residual stream, for a projection that takes 8 bits with a scale each 128.
        dict(name="norm_prompt_8bit", op="norm", dtype="bf16", t=8192, h=1, d=2048, gap=0, add=True,
             out="e4m3", group=128, unit=False),
        # The norms of a prompt's query heads, read from the projection's output, odd token count.
        dict(name="norm_heads", op="norm", dtype="fp16", t=4097, h=16, d=256, gap=4, add=False,
             out="fp16", group=0, unit=True),
        # The queries, keys and values of one token: 16 and 2 x 2 heads of 256 from 2048 features.
        dict(name="proj_decode_one", op="linear", x="bf16", out="bf16", t=1, k=2048, o=5120, group=64,
             xgroup=0, scale="fp16"),
        # A decode batch's heads back to the stream, activations in 8 bits, an odd number of rows.
        dict(name="proj_batch_8bit", op="linear", x="e4m3", out="bf16", t=37, k=4096, o=2047, group=64,
             xgroup=128, scale="bf16"),
        # A small batch's logits over a vocabulary, which the sampling wants in fp32.
        dict(name="proj_vocabulary", op="linear", x="bf16", out="fp32", t=8, k=2048, o=130001, group=64,
             xgroup=0, scale="fp16"),
        # Four continuations of one prompt, a token each: the smallest shared batch.
        dict(name="shared_few", op="shared", dtype="bf16", groups="4", prefix=1501, tail=37, nq=1,
             hq=16, hk=2, d=256, page=16),
        # Many samples of one long prompt, which is read once for all of them.
        dict(name="shared_many", op="shared", dtype="bf16", groups="48", prefix=16384, tail=700, nq=1,
             hq=16, hk=2, d=256, page=64),
        # A server's batch: groups of several sizes, a lone sequence, three drafted tokens each.
        dict(name="shared_groups", op="shared", dtype="fp16", groups="7,1,16,2,31", prefix=6001, tail=515,
             nq=3, hq=24, hk=8, d=128, page=48),
        # One user's next token from a vocabulary's logits with the usual settings.
        dict(name="sample_one", op="sample", dtype="fp32", b=1, v=130001, mode="usual"),
        # A decode batch in which every row has settings of its own, greedy ones among them.
        dict(name="sample_mixed", op="sample", dtype="bf16", b=48, v=65521, mode="mixed"),
        # Many rollouts at once: temperature and the nucleus over the whole vocabulary.
        dict(name="sample_rollouts", op="sample", dtype="fp32", b=256, v=131072, mode="nucleus"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "shared", "sample"])
    dt = rng.choice(["bf16", "fp16"])
    if op == "norm":
        d = rng.choice([64, 128, 256, 512, 2048, 4096, _log(rng, 17, 8192)])
        h = rng.choice([1, 1, rng.randint(2, 32)])
        t = min(_log(rng, 1, 16384), max(1, 12_000_000 // (h * d)))
        out = rng.choice([dt, dt, "fp32", "e4m3", "int8"])
        group = rng.choice([g for g in (0, 64, 128) if g == 0 or d % g == 0]) if out in _TOP else 0
        return dict(op="norm", dtype=dt, t=t, h=h, d=d, gap=rng.randint(0, 3) if h > 1 else 0,
                    add=h == 1 and rng.random() < 0.7, out=out, group=group, unit=rng.random() < 0.5)
    if op == "linear":
        group = rng.choice([64, 64, 128])
        k = group * rng.randint(1, 4096 // group)
        o = _log(rng, 1, min(130000, 230_000_000 // k))
        x = rng.choice([dt, dt, "e4m3", "int8"])
        return dict(op="linear", x=x, out=rng.choice(["bf16", "fp16", "fp32"]) if x in _TOP
                    else rng.choice([dt, "fp32"]), t=min(_log(rng, 1, 64), 1 + 6_000_000_000 // (k * o)),
                    k=k, o=o, group=group,
                    xgroup=rng.choice([0, group]) if x in _TOP else 0, scale=rng.choice(["fp16", "bf16"]))
    if op == "shared":
        hk, d, g = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 8])
        groups = [_log(rng, 1, 48) for _ in range(rng.randint(1, 6))]
        n, nq = sum(groups), rng.choice([1, 1, rng.randint(2, 5)])
        # keys a sequence: the plain form holds them all, and each is met by every query
        most = min(25_000_000, 3_000_000_000 // (nq * g)) // (n * hk * d)
        prefix = max(8, min(_log(rng, 16, 16384), most * 3 // 4))
        tail = max(nq, min(_log(rng, 1, 1000), most // 4))
        return dict(op="shared", dtype=dt, groups=",".join(map(str, groups)), prefix=prefix, tail=tail,
                    nq=nq, hq=hk * g, hk=hk, d=d, page=rng.choice([16, 32, 48, 64, 128]))
    v = _log(rng, 100, 200000)
    return dict(op="sample", dtype=rng.choice([dt, "fp32", "fp32"]), b=min(_log(rng, 1, 256), 33_000_000 // v),
                v=v, mode=rng.choice(["usual", "mixed", "nucleus"]))


# ------------------------------------------------------------- what a case is
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, dt, *shape):
    return torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _members(c):
    return [int(x) for x in c["groups"].split(",")]


def _shared(c):
    """The keys that each group shares: the first the most."""
    n = len(_members(c))
    return [max(1, c["prefix"] - i * c["prefix"] // (2 * n)) for i in range(n)]


def _lens(c):
    """Context of every sequence, group by group: the shared keys, and own ones from
    the new tokens alone to the longest tail."""
    lens = []
    for m, p in zip(_members(c), _shared(c)):
        lens += [p + c["nq"] + (i * 7919 % 97) * (c["tail"] - c["nq"]) // 96 for i in range(m)]
    return lens


def _page_table(c, g):
    """Pages scattered over the cache; a group's whole shared pages are the same for its
    members, a shared page that is not full is each member's own copy."""
    page, rows, at = c["page"], [], 0
    lens = _lens(c)
    width = -(-max(lens) // page) + 1
    for m, p in zip(_members(c), _shared(c)):
        whole = p // page
        first = list(range(at, at + whole))
        at += whole
        for _ in range(m):
            need = -(-lens[len(rows)] // page) - whole
            rows.append(first + list(range(at, at + need)) + [-1] * (width - whole - need))
            at += need
    total = at + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    t = torch.tensor(rows, device="cuda")
    return torch.where(t >= 0, perm[t.clamp(min=0)], -1).contiguous(), total


def _settings(c, g):
    """temperature, top-k, top-p and min-p of every row, and its random number."""
    b = c["b"]
    u = torch.rand(b, generator=g, device="cuda")
    row = torch.arange(b, device="cuda")
    t = 0.6 + 0.1 * (row % 7).float()
    k, p, m = torch.zeros_like(row), torch.ones_like(t), torch.zeros_like(t)
    if c["mode"] == "usual":
        k, p = k + 50, p * 0.95
    elif c["mode"] == "nucleus":
        p = p * 0.9
    else:  # greedy; plain; top-k; nucleus; min-p; all together
        kind = row % 6
        t = torch.where(kind == 0, 0.0, t)
        k = torch.where((kind == 2) | (kind == 5), 20 + row, 0)
        p = torch.where((kind == 3) | (kind == 5), 0.92, 1.0)
        m = torch.where((kind == 4) | (kind == 5), 0.02, 0.0)
    return dict(u=u, temperature=t, top_k=k.to(torch.int32), top_p=p, min_p=m)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] == "norm":
        # the stream has a few features far larger than the rest
        dt = _DT[c["dtype"]]
        x = _randn(g, dt, c["t"], c["h"] + c["gap"], c["d"])
        x[..., :: 97] *= 12.0
        s["x"] = x[:, :c["h"]] if c["h"] > 1 or c["gap"] else x[:, 0]
        s["w"] = _randn(g, torch.float32, c["d"]).mul_(0.2).add_(0.0 if c["unit"] else 1.0).to(dt)
        if c["add"]:
            s["r"] = _randn(g, dt, c["t"], c["d"]).mul_(3.0)
        return s
    if c["op"] == "linear":
        # weights N(0, 0.02) as their groups' least value and steps of a 15th of their range
        ng = c["k"] // c["group"]
        s["codes"] = torch.randint(0, 256, (c["o"], c["k"] // 2), dtype=torch.uint8, device="cuda", generator=g)
        low = _randn(g, torch.float32, c["o"], ng).mul_(0.006).sub_(0.048)
        s["scale"] = (low.abs() / 7.5).to(_DT[c["scale"]])
        s["bias"] = low.to(_DT[c["scale"]])
        x = _randn(g, torch.float32, c["t"], c["k"])
        s["x_scale"] = None
        if c["x"] in _TOP:
            xg = c["xgroup"] or c["k"]
            y = x.view(c["t"], -1, xg)
            s["x_scale"] = (y.abs().amax(-1) / _TOP[c["x"]]).contiguous()
            y = y / s["x_scale"][..., None]
            x = (y.round() if c["x"] == "int8" else y).view(c["t"], c["k"])
        s["x"] = x.to(_DT[c["x"]])
        return s
    if c["op"] == "shared":
        dt, lens = _DT[c["dtype"]], _lens(c)
        m = _members(c)
        s["table"], total = _page_table(c, g)
        s["cu"] = _i32([i * c["nq"] for i in range(len(lens) + 1)])
        s["kv_len"] = _i32(lens)
        s["cu_group"] = _i32([0] + np.cumsum(m).tolist())
        s["shared"] = _i32(_shared(c))
        own_keys = [n - p for n, p in zip(lens, [p for k, p in zip(m, _shared(c)) for _ in range(k)])]
        s["hints"] = dict(max_q=c["nq"], max_group=max(m) * c["nq"], max_shared=max(_shared(c)),
                          max_tail=max(own_keys))
        s["max_kv"] = max(lens)
        pool = _randn(g, dt, 2, total, c["page"], c["hk"], c["d"])
        s["k"], s["v"] = pool[0], pool[1]
        # what a group shares in a page that is not full lies in each member's copy of it
        at = 0
        for n, p in zip(m, _shared(c)):
            part, whole = p % c["page"], p // c["page"]
            if part:
                ids = s["table"][at:at + n, whole].long()
                pool[:, ids, :part] = pool[:, ids[:1], :part]
            at += n
        # queries that give peaked scores; behind a sequence's end are no numbers
        s["q"] = _randn(g, dt, len(lens) * c["nq"], c["hq"], c["d"]).mul_(2.0)
        last = s["table"].gather(1, ((s["kv_len"] - 1) // c["page"]).long()[:, None])[:, 0].long()
        behind = torch.arange(c["page"], device="cuda")[None] > ((s["kv_len"] - 1) % c["page"])[:, None]
        bad = torch.zeros(total, c["page"], dtype=torch.bool, device="cuda")
        bad[last] = behind
        pool.masked_fill_(bad[None, :, :, None, None], float("nan"))
        s["scale"] = c["d"] ** -0.5
        return s
    # a row's logits: most of the vocabulary far down, a few likely tokens
    x = _randn(g, torch.float32, c["b"], c["v"]).mul_(2.5)
    hot = torch.randint(0, c["v"], (c["b"], 12), device="cuda", generator=g)
    x.scatter_add_(1, hot, torch.rand(c["b"], 12, device="cuda", generator=g).mul_(12.0))
    s["logits"] = x.to(_DT[c["dtype"]])
    s.update(_settings(c, g))
    return s


# ---------------------------------------------------------------- plain forms
def _dequantised(q, scale, group, dt):
    """What 8-bit values and their scales stand for, in the stream's type."""
    y = q.float().unflatten(-1, (-1, group)) * scale[..., None]
    return y.flatten(-2).to(dt)


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if c["add"]:
        h = h + s["r"].float()
    w = s["w"].float() + (1.0 if c["unit"] else 0.0)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + _EPS) * w
    dt = _DT[c["dtype"]]
    out = [h.to(dt)] if c["add"] else []
    if c["out"] not in _TOP:
        return [y.to(_DT[c["out"]])] + out
    group = c["group"] or c["d"]
    z = y.unflatten(-1, (-1, group))
    scale = z.abs().amax(-1) / _TOP[c["out"]]
    z = z / torch.where(scale > 0, scale, 1.0)[..., None]
    z = (z.round() if c["out"] == "int8" else z).flatten(-2).to(_DT[c["out"]])
    return [_dequantised(z, scale, group, dt), scale] + out


def _plain_linear(s):
    c = s["case"]
    w = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).view(c["o"], -1, c["group"]).float()
    w = (w * s["scale"].float()[..., None] + s["bias"].float()[..., None]).view(c["o"], c["k"])
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = (x.view(c["t"], s["x_scale"].shape[1], -1) * s["x_scale"][..., None]).view(c["t"], c["k"])
    return torch.matmul(x, w.T).to(_DT[c["out"]])


def _plain_shared(s):
    c = s["case"]
    q, table, kvl = s["q"], s["table"].long(), s["kv_len"].long()
    dev, hk, g, n, nq = q.device, c["hk"], c["hq"] // c["hk"], len(_lens(c)), c["nq"]
    j = torch.arange(s["max_kv"], device=dev)
    held = j[None] < kvl[:, None]
    at = torch.where(held, table[:, j // c["page"]], 0)
    zero = torch.zeros((), device=dev)
    k = torch.where(held[..., None, None], s["k"][at, j % c["page"]].float(), zero)
    x = q.float().view(n, nq, hk, g, c["d"]).permute(0, 2, 1, 3, 4).reshape(n, hk, nq * g, c["d"])
    score = torch.matmul(x, k.permute(0, 2, 3, 1)) * s["scale"]
    del k
    pos = (kvl - nq)[:, None] + torch.arange(nq, device=dev)[None]
    see = (j[None, None] <= pos[..., None])[:, None, :, None].expand(-1, 1, -1, g, -1).reshape(n, 1, nq * g, len(j))
    score.masked_fill_(~see, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where(held[..., None, None], s["v"][at, j % c["page"]].float(), zero)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total
    lse = (total.log() + top)[..., 0]
    o = o.view(n, hk, nq, g, c["d"]).permute(0, 2, 1, 3, 4).reshape(n * nq, c["hq"], c["d"])
    return o.to(q.dtype), lse.view(n, hk, nq, g).permute(0, 2, 1, 3).reshape(n * nq, c["hq"])


def _plain_sample(s):
    """In 64 bits: a token next to a border depends on the sums' last bits."""
    z, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = t[:, 0] == 0
    rank = torch.arange(z.shape[1], device=z.device)[None]
    w = torch.exp((z - z[:, :1]) / torch.where(t > 0, t, 1.0))
    k = s["top_k"][:, None]
    w = torch.where((k > 0) & (rank >= k), 0.0, w)
    p = s["top_p"].double()[:, None]
    upto = w.cumsum(1)
    w = torch.where((p < 1) & (upto - w >= p * upto[:, -1:]), 0.0, w)
    w = torch.where(w < s["min_p"].double()[:, None], 0.0, w)
    w = torch.where(greedy[:, None] & (rank > 0), 0.0, w)
    kept = torch.zeros_like(w).scatter_(1, order, w)
    upto = kept.cumsum(1)
    total = upto[:, -1:]
    token = (upto <= s["u"].double()[:, None] * total).sum(1)
    return token.to(torch.int32), (kept.gather(1, token[:, None]) / total).log()[:, 0].float()


# ----------------------------------------------------------------------- run
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "linear": _plain_linear, "shared": _plain_shared,
                "sample": _plain_sample}[c["op"]](s)
    import sparse_moe_bit_gb300 as M
    if c["op"] == "norm":
        out = M.rms_norm(s["x"], s["w"], residual=s.get("r"), eps=_EPS, unit_offset=c["unit"],
                         out_dtype=_DT[c["out"]], group=c["group"])
        if c["out"] not in _TOP:
            return [out[0], out[1]] if c["add"] else [out]
        return [_dequantised(out[0], out[1], c["group"] or c["d"], _DT[c["dtype"]]), *out[1:]]
    if c["op"] == "linear":
        return M.linear4(s["x"], s["codes"], s["scale"], s["bias"], x_scale=s["x_scale"],
                         out_dtype=_DT[c["out"]])
    if c["op"] == "shared":
        return M.paged_attention_shared(s["q"], s["k"], s["v"], s["table"], s["cu"], s["kv_len"], s["cu_group"],
                                        s["shared"], scale=s["scale"], return_lse=True, **s["hints"])
    return M.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                    top_p=s["top_p"], min_p=s["min_p"], return_logprobs=True)


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "norm":
        n, e = c["t"] * c["h"] * c["d"], _SIZE[c["dtype"]]
        scales = n // (c["group"] or c["d"]) * 4 if c["out"] in _TOP else 0
        return dict(bytes=n * (e * (3 if c["add"] else 1) + _SIZE[c["out"]]) + scales + e * c["d"],
                    flops=n * (5 if c["add"] else 4))
    if c["op"] == "linear":
        x = c["t"] * c["k"] * _SIZE[c["x"]] + (c["t"] * c["k"] // (c["xgroup"] or c["k"]) * 4 if c["x"] in _TOP else 0)
        return dict(bytes=c["o"] * (c["k"] // 2 + c["k"] // c["group"] * 4) + x + c["t"] * c["o"] * _SIZE[c["out"]],
                    flops=2 * c["t"] * c["o"] * c["k"])
    if c["op"] == "shared":
        lens, nq = _lens(c), c["nq"]
        keys = sum(lens) - sum((m - 1) * p for m, p in zip(_members(c), _shared(c)))
        pairs = sum(nq * n - nq * (nq - 1) // 2 for n in lens)
        t, e = len(lens) * nq, _SIZE[c["dtype"]]
        return dict(bytes=2 * e * keys * c["hk"] * c["d"] + 2 * e * t * c["hq"] * c["d"] + 4 * t * c["hq"],
                    flops=4 * pairs * c["hq"] * c["d"])
    return dict(bytes=c["b"] * (c["v"] * _SIZE[c["dtype"]] + 28), flops=3 * c["b"] * c["v"])


# --------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits, row by row or sequence by sequence."""
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        outs = []
        for at in range(0, c["t"], 1024):
            h = s["x"][at:at + 1024].double()
            if c["add"]:
                h = h + s["r"][at:at + 1024].double()
            norm = (torch.linalg.vector_norm(h, dim=-1, keepdim=True) ** 2 / c["d"] + _EPS).sqrt()
            y = h / norm * (s["w"].double() + (1 if c["unit"] else 0))
            if c["out"] in _TOP:
                z = y.reshape(*y.shape[:-1], -1, c["group"] or c["d"])
                scale = z.abs().max(-1, keepdim=True).values / _TOP[c["out"]]
                z = z / scale
                # a step of the type at z: whole numbers, or four significant bits down to 2^-9
                step = 1.0 if c["out"] == "int8" else torch.exp2(torch.floor(torch.log2(z.abs())).clamp(min=-6) - 3)
                z = torch.round(z / step) * step * scale
                outs.append([z.reshape(y.shape), scale[..., 0]] + ([h] if c["add"] else []))
            else:
                outs.append([y] + ([h] if c["add"] else []))
        return [torch.cat(x) for x in zip(*outs)]
    if c["op"] == "linear":
        x = s["x"].double()
        if s["x_scale"] is not None:
            x = x * s["x_scale"].double().repeat_interleave(c["k"] // s["x_scale"].shape[1], 1)
        out = []
        for at in range(0, c["o"], 8192):
            code = s["codes"][at:at + 8192]
            w = torch.empty(code.shape[0], c["k"], dtype=torch.float64, device=code.device)
            w[:, 0::2], w[:, 1::2] = code % 16, code // 16
            rep = lambda a: a[at:at + 8192].double().repeat_interleave(c["group"], 1)
            out.append(x @ (w * rep(s["scale"]) + rep(s["bias"])).T)
        return torch.cat(out, 1)
    if c["op"] == "shared":
        outs, lses, nq, g = [], [], c["nq"], c["hq"] // c["hk"]
        for n, kv in enumerate(_lens(c)):
            j = torch.arange(kv, device="cuda")
            row = s["table"][n].long()[j // c["page"]]
            k, v = (s[a][row, j % c["page"]].double() for a in ("k", "v"))
            q = s["q"][n * nq:(n + 1) * nq].double()
            z = torch.einsum("qhd,jhd->hqj", q, k.repeat_interleave(g, 1)) * s["scale"]
            z = z.masked_fill(j > torch.arange(kv - nq, kv, device="cuda")[:, None], -math.inf)
            l = torch.logsumexp(z, -1)
            outs.append(torch.einsum("hqj,jhd->qhd", torch.exp(z - l[..., None]), v.repeat_interleave(g, 1)))
            lses.append(l.T)
        return torch.cat(outs), torch.cat(lses)
    # whole sorts in numpy: a fraction of a second for a million logits
    z = s["logits"].double().cpu().numpy()
    p = {k: s[k].cpu().numpy().astype(np.float64) for k in ("u", "temperature", "top_k", "top_p", "min_p")}
    tokens, logs = [], []
    for b in range(c["b"]):
        if p["temperature"][b] == 0:
            tokens.append(int(np.argmax(z[b])))
            logs.append(0.0)
            continue
        w = np.exp((z[b] - z[b].max()) / p["temperature"][b])
        order = np.argsort(-z[b], kind="stable")
        if p["top_k"][b] > 0:
            order = order[:int(p["top_k"][b])]
        if p["top_p"][b] < 1:
            upto = np.cumsum(w[order])
            order = order[:np.searchsorted(upto, p["top_p"][b] * upto[-1], side="left") + 1]
        kept = np.sort(order[w[order] >= p["min_p"][b]])
        upto = np.cumsum(w[kept])
        at = min(np.searchsorted(upto, p["u"][b] * upto[-1], side="right"), len(kept) - 1)
        tokens.append(int(kept[at]))
        logs.append(math.log(w[kept[at]] / upto[-1]))
    return (torch.tensor(tokens, dtype=torch.int32), torch.tensor(logs, dtype=torch.float64))
