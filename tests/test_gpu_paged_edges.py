"""Narrow cases of the paged-cache calls (include/paged.h) on the GPU."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from tests.paged_cases import attention_reference, check_attention, make_batch

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


@pytest.mark.parametrize("new,kv", [([1], [5000]), ([40], [300]), ([30], [9000])])
def test_given_stream_does_not_write_where_the_current_one_still_works(new, kv):
    """A block let go of on the current stream while its work is still queued there:
    outputs and workspaces of a call on another stream must not be made of it."""
    b = make_batch(2, new, kv, 16, 1, 128, BF, 4, device="cuda")
    names = ("q", "k", "v", "table", "cu", "kv_len")
    f = torch.ones(8, dtype=torch.float64, device="cuda")
    pos = torch.arange(new[0], dtype=torch.int32, device="cuda")
    want = M.paged_attention(*(b[x] for x in names), return_lse=True)
    turned = M.rope(b["q"], pos, f)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty_like(want[0]) for _ in range(3)] + [torch.empty_like(want[1])]
    blocks += [torch.empty(40 << 20, dtype=torch.uint8, device="cuda")]
    at = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in blocks]
    torch.cuda._sleep(20_000_000)            # some 10 ms
    for t in blocks:
        t.fill_(7)
    del blocks, t
    o, lse = M.paged_attention(*(b[x] for x in names), return_lse=True, stream=st)
    y = M.rope(b["q"], pos, f, stream=st)
    for t in (o, lse, y):
        assert not any(a <= t.data_ptr() < z for a, z in at)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(y, turned)
    assert M.paged_device_error() == 0


@pytest.mark.parametrize("nq", [1, 30])
def test_tokens_outside_every_sequence_leave_no_trace(nq):
    """No token belongs to a sequence: nothing is written but the workspace, and
    that not after the call."""
    b = make_batch(3, [nq], [9000], 16, 1, 128, BF, 4, device="cuda")
    b["cu"].fill_(nq)
    out = torch.full_like(b["q"], 5.0)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for i in range(20):
        M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], max_q=nq,
                          max_kv=9000, out=out, workspace=ws)
        ws.fill_(i)
    torch.cuda.synchronize()
    assert torch.all(ws == 19) and torch.all(out == 5)
    assert M.paged_device_error() == 0


@pytest.mark.parametrize("page,width", [(16, 3), (1, 7)])
def test_append_past_the_table_row_leaves_the_cache_alone(page, width):
    """More tokens than a row of the table has pages for: those that fit go where
    they belong, the rest nowhere, and an error bit says so."""
    cap = page * width
    b = make_batch(4, [5, 2], [cap, 2], page, 2, 64, BF, 4, device="cuda", width=width)
    b["kv_len"] = torch.tensor([cap + 3, cap + 1000], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(7, h, 64, device="cuda").to(BF) for h in (4, 2, 2))
    f = torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64, device="cuda")
    kp, vp = b["k"].clone(), b["v"].clone()
    y = M.rope_append(q, k, v, kp, vp, b["table"], b["cu"], b["kv_len"], f)
    assert M.paged_device_error() == M.PAGED_DEVERR_LENGTH
    pos = torch.tensor([cap - 2, cap - 1, cap, cap + 1, cap + 2, cap + 998, cap + 999],
                       dtype=torch.int32, device="cuda")
    assert torch.equal(y, M.rope(q, pos, f))
    turned = M.rope(k, pos, f)
    for i, p in ((0, cap - 2), (1, cap - 1)):
        pg = b["table"][0, p // page].long()
        assert torch.equal(kp[pg, p % page], turned[i]) and torch.equal(vp[pg, p % page], v[i])
        kp[pg, p % page], vp[pg, p % page] = b["k"][pg, p % page], b["v"][pg, p % page]
    assert torch.equal(kp, b["k"]) and torch.equal(vp, b["v"])
    assert M.paged_device_error() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq,kv", [(1, 50), (1, 5000), (40, 90), (40, 128), (30, 9000)])
def test_nan_queries_show_in_output_and_lse(nq, kv, d):
    """A query that is not a number gives an output and an lse that are not, in one
    piece or split over the keys, and no other row does."""
    b = make_batch(5, [nq], [kv], 16, 1, d, BF, 2, device="cpu")
    b["q"][nq - 1, 1, 7] = float("nan")
    b = {n: t.cuda() for n, t in b.items()}
    o, lse = M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], max_q=nq,
                               max_kv=kv, return_lse=True)
    want = torch.zeros(nq, 2, dtype=torch.bool, device="cuda")
    want[nq - 1, 1] = True
    assert torch.equal(torch.isnan(lse), want)
    assert torch.equal(torch.isnan(o).all(-1), want) and torch.equal(torch.isnan(o).any(-1), want)
    assert M.paged_device_error() == 0


@pytest.mark.parametrize("few", [True, False], ids=["rows", "chunk"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_fp16_keeps_the_tail_behind_a_sink(d, few):
    """One key that takes nearly all of the weight and 20,000 that are 17.4 nats
    below it, each less than half of fp16's smallest step: together they are the
    whole result (the key's value is 0).  So many items that no key is split off."""
    kv, page = 20_000, 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, nq = (4 * sms, 1) if few else (sms, 256)
    pages = -(-kv // page)
    k = torch.zeros(pages, page, 1, d, dtype=FP, device="cuda")
    k[0, 0, 0, 0] = 1.0
    v = torch.full((pages, page, 1, d), 1.0, dtype=FP, device="cuda")
    v[0, 0] = 0.0
    q = torch.zeros(n * nq, 1, d, dtype=FP, device="cuda")
    q[:, 0, 0] = 17.4
    z = q[0, 0, 0].double().item()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(n, pages)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda") * nq
    o, lse = M.paged_attention(q, k, v, table, cu, torch.full((n,), kv, dtype=torch.int32, device="cuda"),
                               scale=1.0, causal=False, max_q=nq, max_kv=kv, return_lse=True)
    assert M.paged_device_error() == 0
    tail = (kv - 1) * np.exp(-z)
    ref, l_ref = tail / (1 + tail), z + np.log1p(tail)
    # A weight is off by half a step: 2^-11 of itself, or 2^-25 where it is subnormal, in
    # a scale where the largest is 2^15 (rows) or the reference 2^7 (chunk); the result
    # by 2^-11; fp32 sums of kv terms, the score's fp32 error, the exponential's 2^-21.
    f = ((d + 4) * z + kv) * 2.0 ** -24 + 2.0 ** -21
    small = (kv - 1) * 2.0 ** -(25 + (15 if few else 7))
    err = (o.double() - ref).abs().max().item()
    assert err <= ref * (2 * 2.0 ** -11 + 2 * f) + small, f"off by {err / ref:.3f} of the result"
    assert (lse.double() - l_ref).abs().max().item() <= f + 4 * 2.0 ** -24 * l_ref


@pytest.mark.parametrize("window", [0, 4, 500])
@pytest.mark.parametrize("nq", [3, 60])
def test_tokens_before_position_0_see_nothing(nq, window):
    """A context shorter than the chunk: the tokens that stand before position 0 see
    no key, causal or not."""
    new, kv, causal = [nq, nq, 2], [nq - 2, 0, 40], False
    b = make_batch(6, new, kv, 16, 2, 128, BF, 4, device="cuda", fill=float("nan"))
    o, lse = M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], causal=causal,
                               window=window, max_q=nq, max_kv=max(kv), return_lse=True)
    early = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
    early[:2] = early[nq:2 * nq] = True
    assert torch.all(o[early] == 0) and torch.all(torch.isneginf(lse[early]))
    assert torch.all(torch.isfinite(lse[~early])) and torch.all(torch.isfinite(o))
    ref = attention_reference(b, 128 ** -0.5, causal, window)
    keep = (~early).cpu().numpy()
    for r in ref:
        r[~keep] = np.nan        # (rows that the comparison leaves out)
    check_attention(o, lse, ref, BF, 128, max(kv))


@pytest.mark.parametrize("nq", [2, 12, 60])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 8, 1 << 31, 1 << 40])
def test_windows_larger_than_every_context_hide_nothing(nq, window):
    new, kv = [nq, nq], [max(nq - 9, 1), 100]
    b = make_batch(7, new, kv, 16, 1, 64, BF, 4, device="cuda")
    a = (b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"])
    for causal in (True, False):
        kw = dict(causal=causal, max_q=nq, max_kv=100, return_lse=True)
        for x, y in zip(M.paged_attention(*a, window=window, **kw), M.paged_attention(*a, **kw)):
            assert torch.equal(x, y)


def test_reserve_past_the_largest_length_is_refused():
    """A length that does not fit its int32 counts as a row that is too short."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    page = 1 << 30
    refs, table, lens = i32(1, 1, 0, 0), i32(0, 1, -1, -1)[None].clone(), i32(2 ** 31 - 10)
    keep = refs.clone(), table.clone(), lens.clone()
    moves, status = M.pages_reserve(refs, table, lens, i32(10), page)
    assert status.tolist() == [0, 1] and moves.tolist() == [[-1, -1]]
    assert torch.equal(refs, keep[0]) and torch.equal(table, keep[1]) and torch.equal(lens, keep[2])
    moves, status = M.pages_reserve(refs, table, lens, i32(9), page)
    assert status.tolist() == [0, 0] and lens.tolist() == [2 ** 31 - 1]


@pytest.mark.parametrize("page", [16, 64, 6])
@pytest.mark.parametrize("d,dtype", [(64, FP), (128, BF), (256, BF)])
@pytest.mark.parametrize("nq,window", [(1, 40), (3, 129), (70, 33), (130, 200)])
def test_keys_before_every_window_may_be_gone(nq, window, d, dtype, page):
    """A sliding window's server gives pages back: what lies before the first query's
    window is NaN, and the pages that hold nothing else have bad numbers."""
    new, kv = [nq, 1], [nq + 500, 450]
    b = make_batch(8, new, kv, page, 2, d, dtype, 4, device="cpu")
    ref = attention_reference(b, d ** -0.5, True, window)
    for n, (q, x) in enumerate(zip(new, kv)):
        first = x - q - window + 1
        for j in range(first // page + 1):
            pg = b["table"][n, j].item()
            rows = slice(0, min(page, first - j * page))
            b["k"][pg, rows] = b["v"][pg, rows] = float("nan")
        b["table"][n, :first // page] = torch.tensor([-1, 1 << 30], dtype=torch.int32).repeat(
            first // page)[:first // page]
    b = {x: t.cuda() for x, t in b.items()}
    o, lse = M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], window=window,
                               max_q=nq, max_kv=max(kv), return_lse=True)
    check_attention(o, lse, ref, dtype, d, max(kv))
    assert M.paged_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 3000])
def test_chunk_split_over_the_keys(window, d, dtype):
    """Few tiles over a long context: parts of the keys, joined, at every head size."""
    new, kv = [30, 41], [6000, 777]
    b = make_batch(9, new, kv, 32, 1, d, dtype, 8, device="cuda", fill=float("nan"))
    ref = attention_reference(b, d ** -0.5, True, window)
    o, lse = M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], window=window,
                               max_q=41, max_kv=6000, return_lse=True)
    check_attention(o, lse, ref, dtype, d, 6000)
    assert M.paged_device_error() == 0


@pytest.mark.parametrize("few", [True, False], ids=["rows", "chunk"])
def test_thousands_of_sequences(few):
    """More sequences than threads that look for them, empty ones among them."""
    rng = np.random.default_rng(10)
    new = [int(x) for x in rng.integers(0, 3, 3001)]
    kv = [int(n + x) if n else int(x) for n, x in zip(new, rng.integers(0, 40, 3001))]
    b = make_batch(10, new, kv, 8, 1, 64, BF, 2, device="cuda", fill=float("nan"))
    ref = attention_reference(b, 0.125)
    o, lse = M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"],
                               max_q=2 if few else 64, max_kv=42, return_lse=True)
    check_attention(o, lse, ref, BF, 64, 42)
    assert M.paged_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("nq", [1, 100])
@pytest.mark.parametrize("e", [10, 20, 23, 24, 25, 26, 27, 28, 31, 40])
@pytest.mark.parametrize("times", [1.0, 1.37, 1.913])
def test_scores_whose_steps_pass_the_weights_range(times, e, nq, dtype):
    """Scores of some 2^e in log2 units, where fp32's steps (2^(e - 23)) are larger than what
    a reference is off by: two keys take all of the weight, the later one 2^8 ahead or
    level, and the result is their common value."""
    kv, d = 300, 64
    b = make_batch(11, [nq], [kv], 16, 1, d, dtype, 1, device="cpu")
    b["q"].zero_(), b["k"].zero_(), b["v"].fill_(1.0)
    b["q"][:, 0, 0], b["q"][:, 0, 1] = 1000.0, 1.0
    for key, more in ((5, 0.0), (200, 7.9e6 * 2.0 ** -e)):
        pg, r = b["table"][0, key // 16].item(), key % 16
        b["k"][pg, r, 0, 0], b["k"][pg, r, 0, 1] = 1000.0, more
        b["v"][pg, r] = 3.0
    b = {x: t.cuda() for x, t in b.items()}
    scale = times * 2.0 ** e / 1e6 * np.log(2.0)
    o, lse = M.paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["kv_len"], scale=scale,
                               causal=False, max_q=nq, max_kv=kv, return_lse=True)
    assert M.paged_device_error() == 0
    # two roundings of the weights that meet one value, one of the result: half a step each
    u = torch.finfo(dtype).eps / 2
    assert (o.double() - 3).abs().max().item() <= 3 * 3 * u + 2.0 ** -18
    low, high = times * 2.0 ** e * np.log(2.0), times * (2.0 ** e + 9) * np.log(2.0)
    assert torch.all(lse >= low * (1 - 2.0 ** -20)) and torch.all(lse <= high * (1 + 2.0 ** -20) + 1)
