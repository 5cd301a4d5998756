"""Edges of include/step.h's operators: quotients on a border between two 8-bit values,
scales below fp32's normal numbers, groups of many warps."""
import numpy as np
import pytest
import torch

import sparse_moe_bit_gb300 as M
from tests.step_cases import values

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
E8, I8 = torch.float8_e4m3fn, torch.int8
TOP = {I8: 127.0, E8: 448.0}


def _norm8(w, out, group):
    """The 8-bit norm of a row of ones, whose n are the weights themselves."""
    w = torch.from_numpy(np.ascontiguousarray(w)).cuda()
    x = torch.ones(1, w.numel(), device="cuda")
    assert torch.equal(M.rms_norm(x, w, eps=0.0)[0], w)
    y, s = M.rms_norm(x, w, eps=0.0, out_dtype=out, group=group)
    return y[0].float().cpu().numpy(), s[0].cpu().numpy()


def _to8(q, out):
    """fp32 to the values of an 8-bit type, ties to even."""
    if out is I8:
        return np.rint(q)
    return torch.from_numpy(q).clamp(-448, 448).to(E8).float().numpy()


@pytest.mark.parametrize("out", [E8, I8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("d,group", [(1024, 128), (1024, 0), (512, 256), (4096, 0), (2048, 16), (255, 51), (64, 0)])
def test_quotients_on_the_borders(out, d, group):
    """Half of the values lie on a border between two of the type's, or a step of fp32
    beside one: y is fp32's quotient rounded, to the last of them."""
    rng = np.random.default_rng(d + group)
    g = group or d
    borders = np.arange(126) + 0.5
    if out is E8:
        all8 = torch.arange(127, dtype=torch.uint8).view(E8).double().numpy()
        borders = (all8[1:] + all8[:-1]) / 2
    for power in (-25, -12, 0, 3, 17, 30):
        w = rng.standard_normal((d // g, g)).astype(np.float32) * np.float32(10.0 ** power)
        scale = np.abs(w).max(1, keepdims=True) / np.float32(TOP[out])
        near = (rng.choice(borders, (d // g, g)).astype(np.float32) * scale).astype(np.float32)
        away = np.where(rng.random(near.shape) < 0.5, np.float32(np.inf), np.float32(-np.inf))
        near = np.where(rng.random(near.shape) < 0.5, near, np.nextafter(near, away))
        put = (rng.random(w.shape) < 0.5) & (np.abs(w) < np.abs(w).max(1, keepdims=True))
        w = np.where(put, near * rng.choice([-1, 1], w.shape), w).astype(np.float32)
        y, s = _norm8(w.reshape(-1), out, group)
        assert np.array_equal(s, np.abs(w).max(1) / np.float32(TOP[out]))
        assert np.array_equal(y.reshape(w.shape), _to8(w / s[:, None], out)), power


@pytest.mark.parametrize("out", [E8, I8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("group", [32, 24, 256])
def test_scales_below_the_normal_numbers(out, group):
    """Groups whose largest magnitude is a few of fp32's smallest steps: no scale is 0 and no
    value past the type's end, so that y * scale is within half a step of n."""
    rng = np.random.default_rng(group)
    tiny = 2.0 ** -149
    for most in (1, 2, 50, 63, 64, 100, 223, 224, 300, 447, 449, 1000, 3000, 100000, 2 ** 23, 2 ** 29, 2 ** 31, 2 ** 33):
        steps = rng.integers(-most, most + 1, 768)
        steps[::group] = most * rng.choice([-1, 1], 768 // group)
        w = (steps * tiny).astype(np.float32)          # (to fp32's 24 bits)
        y, s = _norm8(w, out, group)
        w, s = w.astype(np.float64).reshape(-1, group), s.astype(np.float64)[:, None]
        assert (s > 0).all()
        got = y.astype(np.float64).reshape(w.shape) * s
        half = 0.5 * s if out is I8 else np.maximum(np.abs(w) * 2.0 ** -4, s * 2.0 ** -10)
        # (and the quotient's own rounding to fp32)
        assert np.all(np.abs(got - w) <= half * (1 + 2.0 ** -20)), most
        # to nearest, or up where it is not a normal number
        exact = np.abs(w).max(1, keepdims=True) / TOP[out]
        step = np.maximum(2.0 ** (np.floor(np.log2(exact)) - 23), tiny)
        assert np.all(np.abs(s - exact) <= step) and np.all((s >= exact) | (s >= 2.0 ** -126))
    y, s = _norm8(np.zeros(768, np.float32), out, group)
    assert (y == 0).all() and (s == 0).all()


def test_an_infinite_scale():
    """A weight that takes one value past fp32's end: the scale says so, the others are 0."""
    w = np.ones(256, np.float32)
    w[7] = np.inf
    for out in (E8, I8):
        y, s = _norm8(w, out, 128)
        assert np.isposinf(s[0]) and s[1] == np.float32(1.0) / np.float32(TOP[out])
        assert (np.delete(y[:128], 7) == 0).all() and (y[128:] == TOP[out]).all()
        if out is E8:
            assert np.isnan(y[7])


@pytest.mark.parametrize("d,group", [(512, 512), (768, 768), (2304, 768), (2048, 0), (4096, 0), (4096, 1024), (6144, 768),
                                     (8192, 0), (8192, 512), (16384, 0), (24576, 1536), (32768, 0), (32768, 4096)])
@pytest.mark.parametrize("out", [E8, I8], ids=["e4m3", "int8"])
def test_the_largest_of_a_group_in_any_lane(d, group, out):
    """Groups of whole warps, enough rows that a block takes several: the largest magnitude is
    every lane's, chunk's and warp's in turn."""
    rows, vectors = 1300, d // 8
    x = torch.randn(rows, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(d)).to(BF)
    at = torch.arange(rows, device="cuda")
    x[at, at * 37 % vectors * 8 + at % 8] = 30.0
    x[at, at * 32 % vectors * 8] = -29.0          # a first lane's
    n = values(M.rms_norm(x, out_dtype=FP)).reshape(rows, -1, group or d)
    y, s = M.rms_norm(x, out_dtype=out, group=group)
    want = np.abs(n).max(-1) / TOP[out]
    # (the quotient's rounding, and n's last bit)
    assert np.all(np.abs(values(s) - want) <= 2.0 ** -22 * want)
    got = y.float().double().cpu().numpy().reshape(n.shape) * values(s)[..., None]
    half = 0.5 * want[..., None] if out is I8 else np.maximum(np.abs(n) * 2.0 ** -4, want[..., None] * 2.0 ** -10)
    assert np.all(np.abs(got - n) <= half * (1 + 1e-5) + 2.0 ** -21 * np.abs(n))
