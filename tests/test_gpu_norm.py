"""rms_norm against its fp64 definition."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from oracle import step_oracle as SO
from tests.step_cases import rounded_bar, u_of, values

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def _inputs(shape, dtype, seed=0, residual=True, weight=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    x[..., ::7] *= 9
    r = torch.randn(shape, generator=g) * 3 if residual else None
    w = 1 + 0.3 * torch.randn(shape[-1], generator=g)
    dev = lambda t, dt: None if t is None else t.to(dt).cuda()
    return dev(x, dtype), dev(r, dtype), dev(w, weight or dtype)


def _bar(n, d):
    """fp32: a rounding of s, d additions of squares (half of their error behind the root),
    and the root, the weight's addition and two products."""
    return (d / 2 + 12) * 2.0 ** -24 * np.abs(n) + 1e-37


def check(y, n, d, dtype):
    assert y.dtype is dtype
    bar = _bar(n, d) + rounded_bar(n, dtype) * (1 + 1e-3)
    err = np.abs(values(y) - n)
    assert np.all(err <= bar), f"off by {np.max(err / bar):.3f} of the bar"


def check8(y, scale, n, d, group):
    kind = "e4m3" if y.dtype is torch.float8_e4m3fn else "int8"
    s_ref = SO.scales(n, group, kind)
    s = values(scale)
    assert s.shape == s_ref.shape
    assert np.all(np.abs(s - s_ref) <= (d / 2 + 14) * 2.0 ** -24 * s_ref + 1e-44)
    got = y.float().double().cpu().numpy().reshape(*s.shape, group) * s[..., None]
    n = n.reshape(got.shape)
    # half a step: of e4m3 2^-4 of the value, or 2^-10 below its normal numbers; of int8 half of one
    half = np.maximum(np.abs(n) * 2.0 ** -4, s_ref[..., None] * 2.0 ** -10) if kind == "e4m3" else 0.5 * s_ref[..., None]
    bar = half * (1 + 1e-3) + 3 * (d / 2 + 14) * 2.0 ** -24 * np.abs(n) + 1e-37
    assert np.all(np.abs(got - n) <= bar), f"off by {np.max(np.abs(got - n) / bar):.3f} of the bar"


SHAPES = [(1, 2048), (3, 2048), (700, 2048), (5, 1), (7, 3), (2, 17), (9, 255), (600, 257), (4, 1024), (1300, 1000),
          (3, 4096), (650, 4104), (2, 5001), (2, 8192), (1, 12288), (2, 32768), (1, 32767), (4, 5, 64), (33, 16, 256),
          (300, 4, 128), (2, 3, 80)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
def test_against_the_definition(shape, dtype):
    d = shape[-1]
    x, r, w = _inputs(shape, dtype)
    y, s = M.rms_norm(x, w, residual=r)
    n, total = SO.rms_norm(values(x), values(w), values(r))
    check(y, n, d, dtype)
    assert np.all(np.abs(values(s) - total) <= rounded_bar(total, dtype) + 2.0 ** -24 * np.abs(total))
    y = M.rms_norm(x, w, eps=1e-3, unit_offset=True)
    check(y, SO.rms_norm(values(x), values(w), eps=np.float64(np.float32(1e-3)), offset=1.0)[0], d, dtype)
    check(M.rms_norm(x), SO.rms_norm(values(x))[0], d, dtype)


@pytest.mark.parametrize("out", [BF, HF, FP])
@pytest.mark.parametrize("weight", [BF, FP])
def test_types_of_weight_and_output(out, weight):
    x, r, w = _inputs((37, 520), BF, 1, weight=weight)
    y, _ = M.rms_norm(x, w, residual=r, out_dtype=out)
    check(y, SO.rms_norm(values(x), values(w), values(r))[0], 520, out)


@pytest.mark.parametrize("shape,group", [((1, 2048), 0), ((5, 2048), 128), ((700, 2048), 64), ((700, 2048), 0),
                                         ((3, 2048), 2), ((3, 2048), 1), ((2, 32768), 128), ((2, 32768), 1),
                                         ((6, 255), 0), ((6, 255), 51), ((7, 3), 3), ((7, 3), 1), ((2, 32767), 0),
                                         ((9, 384), 96), ((9, 384), 24), ((640, 768), 192), ((640, 768), 256),
                                         ((11, 4, 256), 64), ((640, 3, 80), 0), ((3, 4104), 8), ((3, 4104), 1026)],
                         ids=str)
@pytest.mark.parametrize("out", [torch.float8_e4m3fn, torch.int8], ids=["e4m3", "int8"])
def test_eight_bits(shape, group, out):
    d = shape[-1]
    x, r, w = _inputs(shape, BF, 2)
    y, scale, s = M.rms_norm(x, w, residual=r, out_dtype=out, group=group)
    n, total = SO.rms_norm(values(x), values(w), values(r))
    assert y.dtype is out and scale.shape == (*shape[:-1], d // (group or d))
    check8(y, scale, n, d, group or d)
    assert np.all(np.abs(values(s) - total) <= rounded_bar(total, BF) + 2.0 ** -24 * np.abs(total))


def test_views_of_a_projection():
    """Heads of one projection's output; outputs into views; unaligned features."""
    g = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn(31, 20, 64, device="cuda", generator=g).to(BF)
    w = torch.randn(64, device="cuda", generator=g).to(BF)
    before = qkv.clone()
    q = qkv[:, 3:11]
    y = M.rms_norm(q, w)
    check(y, SO.rms_norm(values(before[:, 3:11]), values(w))[0], 64, BF)
    assert torch.equal(qkv, before)
    M.rms_norm(q, w, out=q)                          # in place: the neighbours stay
    assert torch.equal(q, y) and torch.equal(qkv[:, :3], before[:, :3]) and torch.equal(qkv[:, 11:], before[:, 11:])
    x = torch.randn(9, 130, device="cuda", generator=g).to(BF)[:, 1:100]
    out = torch.full((9, 260), 7.0, dtype=BF, device="cuda")
    M.rms_norm(x, out=out[:, 3:102])
    check(out[:, 3:102], SO.rms_norm(values(x))[0], 99, BF)
    assert (out[:, :3] == 7).all() and (out[:, 102:] == 7).all()


def test_residual_in_place():
    x, r, w = _inputs((70, 2048), BF, 3)
    y, s = M.rms_norm(x, w, residual=r)
    for target in ("residual", "x"):
        a, b = x.clone(), r.clone()
        y2, s2 = M.rms_norm(a, w, residual=b, sum_out=b if target == "residual" else a)
        assert torch.equal(y2, y) and torch.equal(s2, s)
        assert s2.data_ptr() == (b if target == "residual" else a).data_ptr()
        assert torch.equal(a if target == "residual" else b, x if target == "residual" else r)


@pytest.mark.parametrize("rows,d", [(9001, 384), (5003, 1000), (3001, 2048), (1999, 4096), (1203, 8192), (611, 16384),
                                    (3001, 301), (1300, 4103)])
def test_many_rows_of_a_block(rows, d):
    """A block reads its next row before it has written one, in place too."""
    x, r, w = _inputs((rows, d), BF, 4)
    n, total = SO.rms_norm(values(x), values(w), values(r))
    y, s = M.rms_norm(x, w, residual=r)
    check(y, n, d, BF)
    assert np.all(np.abs(values(s) - total) <= rounded_bar(total, BF) + 2.0 ** -24 * np.abs(total))
    z, scale, s2 = M.rms_norm(x, w, residual=r, out_dtype=torch.int8)
    check8(z, scale, n, d, d)
    assert torch.equal(s2, s)
    a, b = x.clone(), r.clone()
    y2, _ = M.rms_norm(a, w, residual=b, out=a, sum_out=b)
    assert torch.equal(a, y) and torch.equal(b, s) and y2.data_ptr() == a.data_ptr()
    y3 = M.rms_norm(x, w)
    M.rms_norm(x, w, out=x)
    assert torch.equal(x, y3)


def test_zeros_nan_and_infinity():
    x = torch.ones(6, 256, dtype=BF, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4, :128] = 0
    y = M.rms_norm(x, eps=1e-6)
    assert (y[1] == 0).all() and y[2].isnan().all() and y[3, 200].isnan() and (y[3, :200] == 0).all()
    for dt in (torch.float8_e4m3fn, torch.int8):
        q, s = M.rms_norm(x, out_dtype=dt, group=128)
        back = q.float() * s.repeat_interleave(128, 1)
        assert (back[1] == 0).all() and (s[1] == 0).all() and (s[4, 0] == 0) and (back[4, :128] == 0).all()
        assert (~s[2].isfinite()).all() and back[2].isnan().all() and not s[3, 1].isfinite()
        check8(q[:1], s[:1], values(y.float()[:1]), 256, 128)
    assert M.rms_norm(x[:0]).shape == (0, 256)
    assert M.rms_norm(torch.zeros(3, 0, 8, dtype=BF, device="cuda")).shape == (3, 0, 8)


def test_another_stream_and_a_graph():
    x, r, w = _inputs((40, 512), BF, 4)
    want = M.rms_norm(x, w, residual=r, out_dtype=torch.int8, group=64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = M.rms_norm(x, w, residual=r, out_dtype=torch.int8, group=64, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    y, s = torch.empty_like(x), torch.empty_like(x)
    with torch.cuda.graph(graph):
        M.rms_norm(x, w, residual=r, out=y, sum_out=s)
    for seed in (5, 6):
        x2, r2, _ = _inputs((40, 512), BF, seed)
        x.copy_(x2)
        r.copy_(r2)
        graph.replay()
        check(y, SO.rms_norm(values(x2), values(w), values(r2))[0], 512, BF)
