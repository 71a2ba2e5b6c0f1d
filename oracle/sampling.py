"""Choice of the next token in plain numpy, 64 bits, from the definition over real weights."""
import numpy as np


def keep_set(x, temperature, top_k, top_p, min_p):
    """Kept token ids in ascending order, and the weight of every token."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    with np.errstate(invalid="ignore"):
        w = np.where(x == x.max(), 1.0, np.exp((x - x.max()) / temperature))
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        mass, kept, before = sum(w[i] for i in order), [], 0.0
        for i in order:
            if kept and not before < top_p * mass:
                break
            kept.append(i)
            before += w[i]
        order = kept
    return np.array(sorted(i for i in order if w[i] >= min_p)), w


def sample(x, temperature, top_k, top_p, min_p, u):
    """(id, log probability, margin): margin is how far u lies from the nearest boundary between two tokens."""
    x = np.asarray(x, np.float64)
    clean = np.where(np.isnan(x), -np.inf, x)
    if not (clean > -np.inf).any():
        return -1, -np.inf, 1.0
    if not temperature > 0:
        return int(np.argmax(clean)), 0.0, 1.0
    kept, w = keep_set(x, temperature, top_k, top_p, min_p)
    edge = np.cumsum(w[kept]) / w[kept].sum()
    at = min(int(np.searchsorted(edge, u, side="right")), len(kept) - 1)
    lower = edge[at - 1] if at else -1.0
    upper = edge[at] if at < len(kept) - 1 else 2.0
    return int(kept[at]), float(np.log(w[kept[at]] / w[kept].sum())), float(min(u - lower, upper - u))
