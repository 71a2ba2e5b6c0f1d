"""Residual norms, 4-bit projections and token scores in plain numpy, 64 bits, from their definitions."""
import numpy as np


def normed(v, weight, eps, offset):
    y = v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return y if weight is None else y * (offset + weight)


def residual_norm(x, residual, post=None, pre=None, gate=None, sigmoid=False, scale=1.0, eps=1e-6, offset=0.0):
    """(residual_out, y, size): size bounds what was added up in each element of residual_out."""
    r = np.asarray(residual, np.float64)
    size = np.abs(r)
    if x is not None:
        n = np.asarray(x, np.float64)
        if post is not None:
            n = normed(n, post, eps, offset)
        if gate is not None:
            n = n * (1 / (1 + np.exp(-gate)) if sigmoid else gate)
        r = r + scale * n
        size = size + np.abs(scale * n)
    return r, normed(r, pre, eps, offset), size


def unpacked(codes, scales, group):
    """Weights [out, in] of 4-bit codes and group scales."""
    n, half = codes.shape
    w = np.empty((n, 2 * half))
    for odd in (0, 1):
        c = (codes.astype(np.int64) >> (4 * odd)) & 15
        w[:, odd::2] = np.where(c >= 8, c - 16, c)
    for g in range(scales.shape[1]):
        w[:, g * group:(g + 1) * group] *= np.asarray(scales, np.float64)[:, g:g + 1]
    return w


def linear_q4(x, codes, scales, group, bias=None):
    """(out, size): size is the sum of the products' absolute values."""
    x, w = np.asarray(x, np.float64), unpacked(codes, scales, group)
    out, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        out, size = out + bias, size + np.abs(bias)
    return out, size


def logprobs(x, target, top):
    """(logp, entropy, rank, ids, their logp) of one row."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max()
    if m == -np.inf:
        logs = np.full(len(x), -np.inf)
    else:
        with np.errstate(invalid="ignore"):
            d = np.where(x == m, 0.0, x - m)
        logs = d - np.log(np.exp(d).sum())
    p = np.exp(logs)
    entropy = -(p[p > 0] * logs[p > 0]).sum()
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    ids = [i for i in order[:top] if x[i] > -np.inf]
    fill = top - len(ids)
    lp, rank = (float(logs[target]), order.index(target)) if 0 <= target < len(x) else (0.0, -1)
    return lp, float(entropy), rank, ids + [-1] * fill, [float(logs[i]) for i in ids] + [-np.inf] * fill
