"""Attention step in plain numpy, 64 bits: page tables, norm + rotation, attention of one head over its keys."""
import numpy as np


def tables(ctx, new, table, free, head, page, rows):
    """Returns (table, row_start, seq_len, positions, slots, head) of a step, request by request."""
    table = [list(t) for t in table]
    row_start, positions, slots = [0], [], []
    for r, (c, n) in enumerate(zip(ctx, new)):
        for j in range(-(-c // page), -(-(c + n) // page)):
            table[r][j] = free[head]
            head += 1
        for p in range(c, c + n):
            positions.append(p)
            slots.append(table[r][p // page] * page + p % page)
        row_start.append(row_start[-1] + n)
    pad = rows - len(positions)
    return (np.array(table), np.array(row_start), np.array(ctx) + np.array(new), np.array(positions + [0] * pad),
            np.array(slots + [-1] * pad), head)


def norm_rotate(x, weight, eps, cos, sin, pairs):
    """One head [D]: y = x / sqrt(mean x^2 + eps) * weight (weight None: x), then the rotation by cos, sin [rotary/2]."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * np.asarray(weight, np.float64)
    y = x.copy()
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        y[a] = x[a] * cos[i] - x[b] * sin[i]
        y[b] = x[b] * cos[i] + x[a] * sin[i]
    return y


def attend(q, k, v, pos, scale, window):
    """One query [D] at position pos over keys and values [n, D].  Returns (out, sum of p |v|); zeros when it sees no key."""
    lo = max(0, pos - window + 1) if window else 0
    if pos < 0:
        return np.zeros(v.shape[1]), np.zeros(v.shape[1])
    s = k[lo:pos + 1] @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v[lo:pos + 1], p @ np.abs(v[lo:pos + 1])
