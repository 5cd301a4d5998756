"""sample against its fp64 definition."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from oracle import step_oracle as SO
from tests.step_cases import values

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def check_row(token, logprob, z, u, t=1.0, k=0, p=1.0, m=0.0):
    """The token and its probability, where the definition leaves no doubt; next to a border
    (a part in 2^32 of the sum: the weights are off by 2^-36 of themselves and half of 2^-45
    of the largest each) the neighbours too."""
    zz, w = SO.token_weights(z, t if t > 0 else 1.0)
    if w is None:
        assert token == -1 and (logprob is None or np.isnan(logprob))
        return
    eps = 2.0 ** -32
    want = set()
    for du in (-eps, 0, eps):
        for dp in (-eps, 0, eps) if p < 1 else (0,):
            for dm in (-eps, 0, eps) if m > 0 and m < 1 else (0,):
                want.add(SO.sample(z, min(max(u + du, 0), 1), t, k, p * (1 + dp), m * (1 + dm)))
    assert token in {x[0] for x in want}, (token, want, u)
    if logprob is not None:
        ref = [x[1] for x in want if x[0] == token]
        assert min(abs(logprob - x) for x in ref) <= 2.0 ** -20 * (1 + abs(ref[0]))


def run(z, u, t=1.0, k=0, p=1.0, m=0.0):
    zd = z.cuda()
    B = z.shape[0]
    vec = lambda v, dt: torch.as_tensor(v, dtype=dt).expand(B).contiguous().cuda()
    args = [vec(t, FP), vec(k, torch.int32), vec(p, FP), vec(m, FP)]
    u = torch.as_tensor(u, dtype=FP)
    tok, lp = M.sample(zd, u.cuda(), *args, return_logprobs=True)
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy()
    a = [x.cpu().double().numpy() for x in args]
    for b in range(B):
        check_row(tok[b], lp[b], values(z[b]), float(u[b]), a[0][b], int(a[1][b]), a[2][b], a[3][b])
    return tok


def logits(seed, B, V, dtype=FP, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(B, V, generator=g) * scale
    z[:, ::max(V // 7, 1)] += 4
    return z.to(dtype), torch.rand(B, generator=g)


SETTINGS = [dict(), dict(t=0.7), dict(t=0.0), dict(k=1), dict(k=50, t=0.8), dict(p=0.9), dict(p=0.5, t=1.7),
            dict(m=0.05), dict(k=40, p=0.95, m=0.01, t=0.6), dict(p=0.0), dict(k=7, p=0.3), dict(m=1.0)]


@pytest.mark.parametrize("V", [1, 2, 31, 100, 513, 2048, 2049, 5001, 20000])
@pytest.mark.parametrize("kw", SETTINGS, ids=str)
def test_settings(V, kw):
    run(*logits(V, 5, V), **kw)


@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,V", [(1, 130001), (3, 65521), (40, 8191), (300, 700), (2, 360448), (1, 360447)])
def test_sizes(dtype, B, V):
    z, u = logits(B + V, B, V, dtype)
    rows = torch.arange(B)
    run(z, u, t=0.5 + 0.25 * (rows % 4), k=torch.where(rows % 3 == 0, 0, 60), p=torch.where(rows % 2 == 0, 0.9, 1.0),
        m=torch.where(rows % 5 == 4, 0.02, 0.0))
    run(z, u)


def test_ties_go_to_the_lowest_index():
    z = torch.zeros(6, 300)
    z[:, 250] = 1.0
    z[1:, 7] = 1.0
    u = torch.tensor([0.2, 0.2, 0.2, 0.999, 0.999, 0.75])
    tok = run(z, u, t=torch.tensor([0.0, 0.0, 1.0, 1.0, 1.0, 1.0]), k=torch.tensor([0, 0, 1, 1, 2, 2]))
    assert tok.tolist() == [250, 7, 7, 7, 250, 250]
    # all equal: top-k keeps the first ones, top-p the first that reach it
    z = torch.full((5, 4096), -3.5)
    u = torch.tensor([0.0, 0.4999, 0.5, 0.9999, 0.9999])
    tok = M.sample(z.cuda(), u.cuda(), top_k=10).cpu()
    assert tok.tolist() == [0, 4, 5, 9, 9]
    tok = M.sample(z.cuda(), u.cuda(), top_p=0.25).cpu()
    assert tok.tolist() == [0, 511, 512, 1023, 1023]
    tok = M.sample(z.cuda(), u.cuda(), top_p=0.25, top_k=8).cpu()
    assert tok.tolist() == [0, 0, 1, 1, 1]
    assert M.sample(z.cuda(), u.cuda(), min_p=1.0).cpu().tolist() == [0, 2047, 2048, 4095, 4095]


def test_ties_across_the_slices_of_a_row():
    """Quantised logits of a long row: the threshold's key occurs in every CTA's slice."""
    g = torch.Generator().manual_seed(1)
    z = (torch.randn(4, 100003, generator=g) * 2).round()
    u = torch.tensor([0.03, 0.37, 0.71, 0.9999])
    for kw in (dict(k=100), dict(k=5000), dict(p=0.7), dict(p=0.93, k=30000), dict(m=0.3)):
        run(z, u, **kw)


@pytest.mark.parametrize("V", [2049, 9000, 131072])
@pytest.mark.parametrize("scale", [0.01, 0.5, 2.5, 8.0, 30.0])
def test_nuclei_of_all_sizes(V, scale):
    """From one token to nearly all of the row; logits that differ by less than a bin among them."""
    z, u = logits(V, 4, V, FP, scale)
    for p in (1e-6, 0.1, 0.5, 0.9, 0.99, 0.9999, 1 - 2.0 ** -24):
        run(z, u, p=p)
    run(z.to(BF), u, p=torch.tensor([0.3, 0.8, 0.95, 0.999]), m=torch.tensor([0.0, 1e-3, 0.2, 0.0]))


@pytest.mark.parametrize("V", [2100, 50000])
@pytest.mark.parametrize("offset", [-20000.0, -515.0, -30.0, 30.0, 517.0, 1040.0, 3e5])
def test_rows_far_from_zero_wide_ones_and_masked_ones(V, offset):
    """The bins are made before a row's largest logit is known."""
    z, u = logits(V, 5, V)
    z = z + offset
    z[1] = offset + (z[1] - offset) * 12        # wider than the bins of one circle
    z[2, ::3] = float("-inf")
    z[3, 1::2] = torch.finfo(FP).min
    z[4, 5:] = torch.finfo(FP).min              # five tokens are left
    for kw in (dict(p=0.9), dict(p=0.5, t=3.0), dict(k=40), dict(k=1500, p=0.95), dict(p=0.99, t=0.05),
               dict(p=0.7, t=200.0), dict(k=V - 1, p=0.9, t=0.6)):
        run(z, u, **kw)
    run(z.clamp(min=-6e4).to(BF), u, p=0.9)


def test_top_k_of_all_sizes():
    z, u = logits(9, 4, 40000)
    for k in (1, 2, 100, 1000, 2047, 2048, 2049, 3000, 39999, 40000):
        run(z, u, k=k)
        run(z, u, k=k, p=0.8, m=0.001)
    run(z.to(BF), u, k=torch.tensor([3, 300, 1500, 20000]), p=0.97)


def test_few_distinct_logits():
    """Every bin holds one value: a threshold's key is most of its band."""
    g = torch.Generator().manual_seed(12)
    z = torch.randint(0, 12, (5, 30011), generator=g).float() * 0.75
    u = torch.tensor([0.0, 0.21, 0.5, 0.83, 0.9999])
    for kw in (dict(p=0.2), dict(p=0.55, m=0.01), dict(p=0.9), dict(k=1000), dict(k=9000, p=0.5), dict(k=29000)):
        run(z, u, **kw)


def test_special_logits():
    inf, nan = float("inf"), float("nan")
    z = torch.randn(9, 500, generator=torch.Generator().manual_seed(2))
    z[0] = -inf
    z[1] = nan
    z[2, 3:] = -inf
    z[3, 100] = z[3, 400] = inf
    z[4, ::2] = nan
    z[5] = 3e38
    z[5, 9] = -3e38
    z[6] = 0.0
    z[6, 1::2] = -0.0
    z[7, 10] = inf
    z[8, :] = nan
    z[8, 77] = -1e30
    u = torch.full((9,), 0.6)
    for kw in (dict(), dict(t=0.0), dict(k=3), dict(p=0.8), dict(m=0.5), dict(t=inf), dict(k=400, p=0.99, m=1e-6)):
        tok = run(z, u, **kw)
        assert tok[0] == -1 and tok[1] == -1 and tok[8] == 77 and tok[7] == 10
    # -0 and +0 tie
    assert run(z, u, t=0.0)[6] == 0


def test_settings_out_of_range():
    z, u = logits(3, 1, 200)
    one = lambda **kw: M.sample(z.cuda(), u.cuda(), **kw).item()
    nan, plain, top = float("nan"), one(), int(values(z[0]).argmax())
    assert one(temperature=-1.0) == one(temperature=nan) == top
    assert one(top_k=-5) == one(top_k=200) == one(top_k=10 ** 9) == one(top_p=1.5) == one(top_p=nan) == plain
    assert one(min_p=-1.0) == one(min_p=nan) == plain and one(min_p=7.0) == one(top_p=-1.0) == top
    last = M.sample(torch.zeros(4, 50, device="cuda"), torch.tensor([1.0, 2.0, -1.0, nan], device="cuda"))
    assert last.tolist() == [49, 49, 0, 0]
    assert one(temperature=1e-30) == top and one(temperature=1e-42) == top


def test_extreme_temperatures_and_u():
    z, _ = logits(4, 8, 3000)
    u = torch.tensor([0.0, 2.0 ** -24, 1 - 2.0 ** -24, 0.5, 1e-7, 0.25, 0.75, 0.999])
    for t in (1e-3, 0.05, 30.0, 1e6):
        run(z, u, t=t)
        run(z, u, t=t, p=0.6)


def test_rows_do_not_depend_on_the_batch():
    """One row alone (eight CTAs) and among many (fewer) gives one token."""
    z, u = logits(5, 300, 6000)
    kw = dict(temperature=0.9, top_p=0.95, top_k=900)
    whole, lw = M.sample(z.cuda(), u.cuda(), **kw, return_logprobs=True)
    for b in (0, 17, 299):
        t, l = M.sample(z[b:b + 1].cuda(), u[b:b + 1].cuda(), **kw, return_logprobs=True)
        assert t[0] == whole[b] and l[0] == lw[b]
    for _ in range(3):
        assert torch.equal(M.sample(z.cuda(), u.cuda(), **kw), whole)


def test_frequencies():
    """Draws on a grid of u follow the kept distribution: a count is off by one at most."""
    z, _ = logits(6, 1, 64)
    n = 4096
    u = (torch.arange(n) + 0.5) / n
    tok = M.sample(z.expand(n, -1).contiguous().cuda(), u.cuda(), temperature=0.8, top_k=20).cpu().numpy()
    w = np.exp(values(z[0]) / float(np.float32(0.8)))
    w[np.argsort(-values(z[0]), kind="stable")[20:]] = 0
    assert np.all(np.abs(np.bincount(tok, minlength=64) - n * w / w.sum()) <= 1 + 1e-3)


def test_views_numbers_streams_and_graphs():
    z, u = logits(7, 6, 1000, BF)
    big = torch.full((6, 1013), 99.0, dtype=BF, device="cuda")
    big[:, 7:1007] = z.cuda()
    want = M.sample(z.cuda(), u.cuda(), 0.7, 50, 0.9, 0.01)
    assert torch.equal(M.sample(big[:, 7:1007], u.cuda(), 0.7, 50, 0.9, 0.01), want)
    st = torch.cuda.Stream()
    zc, uc = z.cuda(), u.cuda()
    st.wait_stream(torch.cuda.current_stream())
    got = M.sample(zc, uc, 0.7, 50, 0.9, 0.01, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty(6, dtype=torch.int32, device="cuda")
    with torch.cuda.graph(graph):
        M.sample(zc, uc, 0.7, 50, 0.9, 0.01, out=out)
    z2, u2 = logits(8, 6, 1000, BF)
    zc.copy_(z2)
    uc.copy_(u2)
    graph.replay()
    assert torch.equal(out, M.sample(z2.cuda(), u2.cuda(), 0.7, 50, 0.9, 0.01))
    assert M.sample(zc[:0], uc[:0]).shape == (0,)
