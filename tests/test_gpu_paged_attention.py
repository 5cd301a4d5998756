"""Attention over the paged cache (include/paged.h) against its fp64 definition.
Error bounds: tests/paged_cases.py attention_bars()."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from tests.paged_cases import attention_reference, check_attention, make_batch, values

pytestmark = pytest.mark.gpu


def _run(b, **kw):
    kw.setdefault("return_lse", True)
    r = M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], **kw)
    torch.cuda.synchronize()
    return r


def _check(b, new, kv, **kw):
    d = b["q"].shape[2]
    hints = kw.pop("hints", dict(max_q=max(new), max_kv=max(kv)))
    ref = attention_reference(b, kw.get("scale") or d ** -0.5, kw.get("causal", True), kw.get("window", 0))
    o, lse = _run(b, **kw, **hints)
    check_attention(o, lse, ref, b["q"].dtype, d, max(max(kv), 1))
    assert M.paged_device_error() == 0
    return o, lse


BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 3, 8])
def test_decode(d, g, dtype):
    """One new token a sequence, contexts from one key on, ends inside a page."""
    kv = [1, 2, 15, 16, 17, 64, 65, 300, 1027]
    new = [1] * len(kv)
    b = make_batch(d + g, new, kv, 16, 2, d, dtype, 2 * g, device="cuda", fill=float("nan"))
    _check(b, new, kv)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 48, 64, 128, 250])
def test_page_sizes(page):
    new, kv = [1, 2, 5, 40], [200, 129, 333, 97]
    b = make_batch(page, new, kv, page, 2, 128, BF, 6, device="cuda", fill=float("inf"))
    _check(b, new, kv)


@pytest.mark.parametrize("d,dtype", [(64, FP), (128, BF), (256, BF), (256, FP)])
@pytest.mark.parametrize("nq,kv,g", [(2, 50, 8), (5, 5, 4), (16, 300, 2), (17, 129, 1),
                                     (33, 511, 8), (100, 100, 3), (128, 1024, 2), (130, 257, 5),
                                     (64, 64, 24)])
def test_chunks(nq, kv, g, d, dtype):
    b = make_batch(nq + kv, [nq], [kv], 16, 1, d, dtype, g, device="cuda", fill=float("nan"))
    _check(b, [nq], [kv])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 7, 64, 128, 129, 1000])
def test_window(window, d):
    new, kv = [1, 3, 70, 150], [400, 131, 300, 150]
    b = make_batch(window, new, kv, 16, 1, d, BF, 4, device="cuda")
    _check(b, new, kv, window=window)


@pytest.mark.parametrize("window", [0, 40])
def test_not_causal(window):
    new, kv = [1, 20, 64], [33, 300, 140]
    b = make_batch(5, new, kv, 32, 2, 128, BF, 4, device="cuda")
    _check(b, new, kv, causal=False, window=window)


@pytest.mark.parametrize("nq", [1, 4, 150])
def test_rows_that_see_nothing(nq):
    """A context shorter than the chunk (its first tokens stand before position
    0), an empty context and a sequence without new tokens."""
    new, kv = [nq, nq, 0, 2, nq], [max(nq - 3, 0), 0, 50, 2, 130]
    b = make_batch(6, new, kv, 16, 2, 128, BF, 4, device="cuda", fill=float("nan"))
    o, lse = _check(b, new, kv)
    assert torch.all(o[nq:2 * nq] == 0) and torch.all(torch.isneginf(lse[nq:2 * nq]))


@pytest.mark.parametrize("nq", [1, 60])
def test_bad_pages_are_left_out(nq):
    new, kv = [nq, nq], [200, 90]
    b = make_batch(7, new, kv, 16, 1, 64, BF, 4, device="cpu")
    b["table"][0, 3] = -1
    b["table"][0, 5] = 1 << 20
    b["table"][1, 0] = -(1 << 30)
    b = {k: t.cuda() for k, t in b.items()}
    ref = attention_reference(b, 0.125)
    o, lse = _run(b, max_q=nq, max_kv=200)
    check_attention(o, lse, ref, BF, 64, 200)
    assert M.paged_device_error() == M.PAGED_DEVERR_PAGE
    assert M.paged_device_error() == 0


def test_bad_offsets_and_lengths_stay_inside():
    """cu_q out of order and out of range, kv_len past the table: read clamped."""
    b = make_batch(8, [4, 4, 4], [40, 40, 40], 16, 1, 64, BF, 2, device="cpu")
    b["cu"] = torch.tensor([-5, 4, 100, 9], dtype=torch.int32)
    b["kv_len"] = torch.tensor([10 ** 9, -7, 40], dtype=torch.int32)
    b["table"][0] = b["table"][0].clamp(min=0)
    b = {k: t.cuda() for k, t in b.items()}
    ref = attention_reference(b, 0.125)
    o, lse = _run(b)
    check_attention(o, lse, ref, BF, 64, 64)


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("hints", [dict(), dict(max_q=1, max_kv=16), dict(max_q=1000, max_kv=1 << 20),
                                   dict(max_q=1, max_kv=0), dict(max_q=0, max_kv=300)])
def test_hints_bound_nothing(hints, nq):
    new, kv = [1, nq, 2], [700, 900, 33]
    b = make_batch(9, new, kv, 16, 1, 128, BF, 4, device="cuda")
    _check(b, new, kv, hints=hints)


@pytest.mark.parametrize("nq", [1, 50])
def test_strides(nq):
    """Head-major pages inside an array of all layers, queries inside a fused
    projection, a strided output; neighbours stay as they were."""
    new, kv = [nq, 1], [140, 77]
    b = make_batch(10, new, kv, 16, 3, 128, BF, 6, device="cuda")
    P = b["k"].shape[0]
    pool = torch.full((2, 2, P, 3, 16, 128), 7.0, dtype=BF, device="cuda")
    pool[1, 0] = b["k"].transpose(1, 2)
    pool[1, 1] = b["v"].transpose(1, 2)
    x = torch.randn(nq + 1, 10, 128, device="cuda").to(BF)
    x[:, 2:8] = b["q"]
    out = torch.full((nq + 1, 8, 256), 5.0, dtype=BF, device="cuda")
    v = dict(b, q=x[:, 2:8], k=pool[1, 0].transpose(1, 2), v=pool[1, 1].transpose(1, 2))
    assert not v["k"].is_contiguous()
    o, lse = _run(v, max_q=nq, max_kv=140, out=out[:, 1:7, 64:192])
    ref = attention_reference(b, 128 ** -0.5)
    check_attention(o, lse, ref, BF, 128, 140)
    assert torch.all(out[:, 0] == 5) and torch.all(out[:, 7] == 5)
    assert torch.all(out[..., :64] == 5) and torch.all(out[..., 192:] == 5)


@pytest.mark.parametrize("nq", [1, 90])
def test_extreme_scores(nq):
    """Scores far apart (one key takes the weight), and of equal size."""
    b = make_batch(11, [nq], [300], 16, 1, 128, BF, 4, device="cpu")
    b["q"] *= 60
    b = {k: t.cuda() for k, t in b.items()}
    _check(b, [nq], [300])
    b["q"].zero_()
    _check(b, [nq], [300])
    _check(b, [nq], [300], scale=1e-30)


@pytest.mark.parametrize("nq", [1, 70])
def test_maximum_that_keeps_rising(nq):
    """Keys sorted so that the running maximum rises all the way."""
    b = make_batch(12, [nq], [1000], 16, 1, 64, FP, 2, device="cpu")
    ids = b["table"][0, :63].long()
    flat = b["k"][ids].reshape(-1, 64)
    ramp = torch.linspace(-3, 3, flat.shape[0])[:, None]
    b["k"][ids] = (torch.ones(64) * ramp).reshape(63, 16, 1, 64).to(FP)
    b["q"] = torch.ones_like(b["q"]) * 4
    b = {k: t.cuda() for k, t in b.items()}
    _check(b, [nq], [1000])


@pytest.mark.parametrize("new,kv", [([1], [20000]), ([1, 1, 1], [9000, 3, 5001]), ([30], [6000])])
def test_split_over_the_keys_is_deterministic(new, kv):
    b = make_batch(13, new, kv, 64, 1, 256, BF, 8, device="cuda", fill=float("nan"))
    o, lse = _check(b, new, kv)
    for _ in range(3):
        o2, lse2 = _run(b, max_q=max(new), max_kv=max(kv))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_infinite_and_nan_inputs_stay_in_their_rows():
    """A NaN query makes its own rows NaN and no others'."""
    new, kv = [20, 3], [90, 50]
    b = make_batch(14, new, kv, 16, 1, 128, BF, 2, device="cpu")
    b["q"][4, 1, 7] = float("nan")
    b = {k: t.cuda() for k, t in b.items()}
    o, _ = _run(b, max_q=20, max_kv=90)
    bad = torch.isnan(o).any(-1)
    want = torch.zeros_like(bad)
    want[4, 1] = True
    assert torch.equal(bad, want)


def test_other_stream_workspace_and_graph():
    new, kv = [1, 1], [5000, 1200]
    b = make_batch(15, new, kv, 16, 1, 128, BF, 4, device="cuda")
    o, lse = _check(b, new, kv)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    o2 = M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], max_q=1,
                           max_kv=5000, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(o, o2)
    out = torch.zeros_like(o)
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], max_q=1,
                              max_kv=5000, out=out, workspace=ws)
    # the captured call reads its inputs when it runs
    b["kv_len"][0] = 4000
    g.replay()
    torch.cuda.synchronize()
    ref = attention_reference(b, 128 ** -0.5)
    check_attention(out, None, ref, BF, 128, 5000)


def test_largest_stride_offsets_pass_32_bits():
    """A cache whose last page begins past 2^31 elements."""
    P, page, d = 40000, 64, 256
    pool = torch.empty(P, page, 4, d, dtype=BF, device="cuda")   # 5.2 G elements
    b = make_batch(16, [1, 40], [130, 200], page, 4, d, BF, 4, device="cuda")
    old = b["table"].clone()
    n = b["k"].shape[0]
    v = torch.empty_like(pool)
    pool[P - n:], v[P - n:] = b["k"], b["v"]
    big = dict(b, k=pool, v=v, table=torch.where(old >= 0, old + (P - n), old))
    o, lse = _run(big, max_q=40, max_kv=200)
    ref = attention_reference(b, d ** -0.5)
    check_attention(o, lse, ref, BF, d, 200)
