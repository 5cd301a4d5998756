"""linear4 against its fp64 definition."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from oracle import step_oracle as SO
from tests.step_cases import linear4_bar, values, weights4

pytestmark = pytest.mark.gpu
BF, HF, FP, E8, I8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int8


def _x(seed, T, K, dtype, xg=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g)
    if dtype in (BF, HF):
        return x.to(dtype).cuda(), None
    y = x.view(T, -1, xg or K)
    s = y.abs().amax(-1) / (448 if dtype is E8 else 127)
    y = (y / s[..., None]).view(T, K)
    return (y.round() if dtype is I8 else y).to(dtype).cuda(), s.cuda()


def _value(x, xs):
    v = x.float().double().cpu().numpy()
    return v if xs is None else v * np.repeat(values(xs), x.shape[1] // xs.shape[1], 1)


def check(y, x, xs, w, out):
    codes, scale, bias = (t.cpu() for t in w)
    v = _value(x, xs)
    ref = SO.linear4(v, codes.numpy(), values(scale), values(bias))
    bar = linear4_bar(v, codes.numpy(), values(scale), values(bias), ref, out, x.dtype is BF)
    assert y.dtype is out and y.shape == ref.shape
    err = np.abs(values(y) - ref)
    assert np.all(err <= bar), f"off by {np.max(err / bar):.3f} of the bar"


def _case(T, K, O, dtype=BF, out=None, group=64, scale=HF, xg=0, seed=0):
    w = [t.cuda() for t in weights4(seed, O, K, group, scale)]
    x, xs = _x(seed + 1, T, K, dtype, xg)
    y = M.linear4(x, *w, x_scale=xs, out_dtype=out)
    check(y, x, xs, w, out or (dtype if dtype in (BF, HF) else BF))
    return y


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32, 33, 48, 49, 64, 65, 131])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
def test_tokens(T, dtype):
    _case(T, 512, 200, dtype)


@pytest.mark.parametrize("K", [64, 128, 192, 256, 320, 576, 1024, 2048, 2112, 4096])
@pytest.mark.parametrize("O", [1, 15, 16, 17, 129, 1000])
def test_sizes(K, O):
    _case(3, K, O)


@pytest.mark.parametrize("T,K,O", [(1, 2048, 5120), (37, 4096, 2047), (8, 2048, 20001), (64, 4096, 300), (64, 8192, 130),
                                   (50, 6208, 130), (5, 36864, 40), (9, 36864, 17), (1, 128, 40000), (40, 64, 20000)])
def test_splits_of_rows_and_of_k(T, K, O):
    _case(T, K, O)


@pytest.mark.parametrize("dtype", [E8, I8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("T,K,O,xg", [(1, 256, 100, 0), (5, 256, 100, 64), (17, 1024, 70, 128), (37, 4096, 129, 128),
                                      (3, 192, 33, 192), (64, 640, 50, 320), (8, 2048, 4096, 0), (8, 2048, 4096, 64)])
@pytest.mark.parametrize("out", [BF, FP])
def test_eight_bit_activations(dtype, T, K, O, xg, out):
    _case(T, K, O, dtype, out, xg=xg)


@pytest.mark.parametrize("scale", [HF, BF], ids=["fp16", "bf16"])
@pytest.mark.parametrize("K,group", [(512, 64), (512, 128), (512, 256), (512, 512), (576, 192), (320, 64), (320, 320)])
@pytest.mark.parametrize("out", [BF, HF, FP])
def test_scale_types_groups_and_outputs(scale, K, group, out):
    _case(6, K, 77, HF, out, group, scale)


def test_views():
    w = [t.cuda() for t in weights4(3, 90, 256, 64, HF)]
    big, _ = _x(4, 20, 520, BF)
    x = big[3:17:2, 8:264]
    want = M.linear4(x.contiguous(), *w)
    check(want, x, None, w, BF)
    assert torch.equal(M.linear4(x, *w), want)
    assert torch.equal(M.linear4(x[2:3], *w), want[2:3])
    out = torch.full((7, 101), 5.0, dtype=BF, device="cuda")
    M.linear4(x, *w, out=out[:, 4:94])
    assert torch.equal(out[:, 4:94], want) and (out[:, :4] == 5).all() and (out[:, 94:] == 5).all()
    assert M.linear4(x[:0], *w).shape == (0, 90)


def test_rows_do_not_depend_on_the_batch_nor_on_time():
    w = [t.cuda() for t in weights4(5, 3000, 2048, 64, HF)]
    x, _ = _x(6, 8, 2048, BF)
    whole = M.linear4(x, *w)
    for _ in range(3):
        assert torch.equal(M.linear4(x, *w), whole)
    assert all(torch.equal(M.linear4(x[i:i + 1], *w)[0], whole[i]) for i in range(8))


def test_extreme_values():
    """fp16's ends, zeros, infinities and NaN stay in their own rows."""
    w = [t.cuda() for t in weights4(7, 64, 256, 64, HF)]
    x, _ = _x(8, 5, 256, HF)
    x[1] = 0
    x[2] *= 2.0 ** -20
    x[3, 9] = float("inf")
    x[4, 250] = float("nan")
    y = M.linear4(x, *w, out_dtype=FP)
    check(y[:3], x[:3], None, w, FP)
    assert (y[1] == 0).all() and not y[3].isfinite().any() and y[4].isnan().all()
    big = torch.full((1, 256), 60000.0, dtype=HF, device="cuda")
    check(M.linear4(big, *w, out_dtype=FP), big, None, w, FP)


@pytest.mark.parametrize("dtype,xg", [(BF, 0), (HF, 0), (E8, 0), (E8, 64), (I8, 64)], ids=str)
@pytest.mark.parametrize("T,K,O", [(3, 256, 100), (12, 2048, 40)])
def test_a_token_that_is_not_finite_is_alone(dtype, xg, T, K, O):
    """(codes, scales and biases of zero among them)"""
    codes, scale, bias = [t.cuda() for t in weights4(31, O, K, 64, BF)]
    codes[0], scale[1], bias[2] = 0, 0, 0
    scale[3], bias[3] = 0, 0
    x, xs = _x(32, T, K, dtype, xg)
    want = M.linear4(x, codes, scale, bias, x_scale=xs, out_dtype=FP)
    bad = {1: float("nan"), 2: float("inf")}
    for t, v in bad.items():
        if dtype in (BF, HF) or (dtype is E8 and t == 1):
            x[t, K - 5 * t] = v
        else:
            xs[t, -1] = v
    y = M.linear4(x, codes, scale, bias, x_scale=xs, out_dtype=FP)
    assert not torch.isfinite(y[1:3]).any()
    keep = [t for t in range(T) if t not in bad]
    assert torch.equal(y[keep], want[keep])


def test_norm_and_product_in_eight_bits():
    """A layer's entry as it is used: the norm's 8 bits go into the product."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(9, 2048, device="cuda", generator=g).to(BF)
    r = torch.randn(9, 2048, device="cuda", generator=g).to(BF)
    w = [t.cuda() for t in weights4(9, 640, 2048, 64, HF)]
    for dt, step in ((E8, 2.0 ** -4), (I8, None)):
        q, s, _ = M.rms_norm(x, residual=r, out_dtype=dt, group=128)
        y = M.linear4(q, *w, x_scale=s)
        check(y, q, s, w, BF)
        exact = SO.linear4(SO.rms_norm(values(x), None, values(r))[0], w[0].cpu().numpy(), values(w[1]), values(w[2]))
        err = np.linalg.norm(values(y) - exact) / np.linalg.norm(exact)
        assert err < (step or 2.0 ** -6)


def test_another_stream_and_a_graph():
    w = [t.cuda() for t in weights4(10, 300, 4096, 64, HF)]
    x, _ = _x(11, 33, 4096, BF)
    want = M.linear4(x, *w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = [M.linear4(x, *w, stream=st) for _ in range(4)]
    here = [M.linear4(x, *w) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, want) for a in got + here)
    graph, y = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        M.linear4(x, *w, out=y)
    x2, _ = _x(12, 33, 4096, BF)
    x.copy_(x2)
    graph.replay()
    assert torch.equal(y, M.linear4(x2, *w))
