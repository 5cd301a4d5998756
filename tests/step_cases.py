"""Inputs and error bounds shared by the tests of include/step.h's operators."""
import numpy as np
import torch


def u_of(dtype):
    """Largest relative error of one rounding to dtype: half a step."""
    return torch.finfo(dtype).eps / 2


def values(t):
    return t.detach().to(torch.float64).cpu().numpy()


def rounded_bar(x, dtype):
    """Half a step at |x|, the subnormal steps' included."""
    return u_of(dtype) * np.abs(x) + torch.finfo(dtype).tiny * u_of(dtype)


def weights4(seed, O, K, group, dtype):
    """Codes, scales and biases of weights N(0, 0.02): bias the least, scale a 15th of the range."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (O, K // 2), dtype=torch.uint8, generator=g)
    low = torch.randn(O, K // group, generator=g) * 0.006 - 0.048
    return codes, (low.abs() / 7.5).to(dtype), low.to(dtype)


def linear4_bar(x, codes, scale, bias, ref, dtype, bf16):
    """Products exact; a part of 64 sums its products in four steps of 17 terms, each off by at
    most 2^-23 of their magnitudes, then three roundings a part and one a part for the sum.
    (bf16: the codes carry 16, which scale and bias take out again.)"""
    K = x.shape[1]
    off = 16.0 if bf16 else 0.0
    c = np.empty((codes.shape[0], K))
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    rep = K // scale.shape[1]
    mag = np.repeat(np.abs(scale), rep, 1) * (c + 2 * off) + np.repeat(np.abs(bias), rep, 1)
    z = np.abs(x) @ mag.T
    return (4 * 17 + 8 + K // 64) * 2.0 ** -23 * z + rounded_bar(ref, dtype) + 1e-30
