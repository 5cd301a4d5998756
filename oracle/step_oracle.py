"""fp64 definitions of include/step.h's operators, row by row (test infrastructure;
shares no code with the GPU path)."""
import numpy as np

TOP = {"e4m3": 448.0, "int8": 127.0}


def rms_norm(x, weight=None, residual=None, eps=1e-6, offset=0.0):
    """n and s = x + residual; x [..., d]."""
    s = x if residual is None else x + residual
    w = 1.0 if weight is None else weight
    return s / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps) * (w + offset), s


def scales(n, group, kind):
    """The scales of a norm's 8-bit form: [..., d / group]."""
    return np.abs(n.reshape(*n.shape[:-1], -1, group)).max(-1) / TOP[kind]


def weights4(codes, scale, bias):
    """[O, K] of uint8 [O, K / 2] (the even k in the low nibble) and [O, K / group]."""
    c = np.empty((codes.shape[0], codes.shape[1] * 2))
    c[:, 0::2] = codes & 15
    c[:, 1::2] = codes >> 4
    rep = c.shape[1] // scale.shape[1]
    return np.repeat(scale, rep, 1) * c + np.repeat(bias, rep, 1)


def linear4(x, codes, scale, bias):
    return x @ weights4(codes, scale, bias).T


def token_weights(z, temperature):
    """exp((z - max) / temperature), +inf sharing, NaN as -inf; None without a token."""
    z = np.where(np.isnan(z), -np.inf, z)
    top = z.max()
    if top == -np.inf:
        return z, None
    if top == np.inf:
        return z, (z == np.inf).astype(float)
    with np.errstate(over="ignore", invalid="ignore"):
        return z, np.where(np.isneginf(z), 0.0, np.exp((z - top) / temperature))


def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logarithm of its probability) of one row."""
    z, w = token_weights(z, temperature if temperature > 0 else 1.0)
    if w is None:
        return -1, np.nan
    if not temperature > 0:
        return int(np.argmax(z)), 0.0
    order = np.argsort(-z, kind="stable")
    if 0 < top_k < len(z):
        order = order[:top_k]
    if top_p < 1:
        upto = np.cumsum(w[order])
        order = order[:np.searchsorted(upto, top_p * upto[-1], side="left") + 1]
    kept = np.sort(order[(w[order] >= min_p) & (w[order] > 0)])
    upto = np.cumsum(w[kept])
    at = kept[min(np.searchsorted(upto, u * upto[-1], side="right"), len(kept) - 1)]
    return int(at), float(np.log(w[at] / upto[-1]))
