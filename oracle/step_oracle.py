"""fp64 oracle of the serving step (include/kamera_step.h): append, attention, page copies.

NumPy only, from the definitions; no code shared with the library. Rows come and go as
float64 arrays; the pool is [L][pages * page_size][F] rows. Each function also returns the
sums of absolute terms that the tests' error bounds are made of.
"""
import numpy as np


def slots(table, slot0, tokens, page_size):
    """Pool rows of own/prefix tokens 0..tokens-1."""
    at = slot0 + np.arange(tokens, dtype=np.int64)
    return np.asarray(table, dtype=np.int64)[at // page_size] * page_size + at % page_size


def attend(q, keys, values, scale, last):
    """softmax(scale q k^T) v for queries [n][G][dk] of one KV head over keys [T][dk], values [T][dv];
    query i sees keys 0..last[i] (none: zeros and -inf). Returns (out, lse, weighted sum of |v|,
    largest sum of |scale q k| terms of a seen key)."""
    n, g, _ = q.shape
    dv = values.shape[1]
    out, absv = np.zeros((n, g, dv)), np.zeros((n, g, dv))
    lse, terms = np.full((n, g), -np.inf), np.zeros((n, g))
    for i in range(n):
        t = int(last[i]) + 1
        if t <= 0:
            continue
        s = scale * (q[i] @ keys[:t].T)
        terms[i] = np.abs(scale) * (np.abs(q[i]) @ np.abs(keys[:t]).T).max(axis=1)
        m = s.max(axis=1, keepdims=True)
        p = np.exp(s - m)
        total = p.sum(axis=1, keepdims=True)
        out[i] = (p / total) @ values[:t]
        absv[i] = (p / total) @ np.abs(values[:t])
        lse[i] = (m + np.log(total))[:, 0]
    return out, lse, absv, terms


def phases(positions, d_rot, base, sections=(0, 0, 0)):
    """Angles [n][d_rot/2]: positions [n] or [n][3], pair i turning by its section's component."""
    i = np.arange(d_rot // 2)
    theta = float(base) ** (-2.0 * i / d_rot)
    pos = np.asarray(positions, dtype=np.float64)
    if pos.ndim == 1:
        return pos[:, None] * theta
    which = np.repeat(np.arange(3), sections) if any(sections) else np.zeros(d_rot // 2, dtype=int)
    return pos[:, which] * theta


def norm(x, weight, eps):
    """x / sqrt(mean(x^2) + eps) * weight over the last axis."""
    return x / np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + eps) * weight


def rotate(x, phi, gptj=False):
    """(rotated, sums of |terms|): x [n][...][d], phi [n][d/2]; pairs (i, i + d/2), or (2i, 2i + 1)."""
    d = x.shape[-1]
    ia = np.arange(0, d, 2) if gptj else np.arange(d // 2)
    ib = ia + 1 if gptj else ia + d // 2
    phi = phi.reshape(phi.shape[0], *([1] * (x.ndim - 2)), d // 2)
    c, s, a, b = np.cos(phi), np.sin(phi), x[..., ia], x[..., ib]
    y, t = np.empty_like(x), np.empty_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    t[..., ia], t[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    return y, t


def copy_pages(pool, src, dst):
    """pool [L][pages][...] after page dst[i] took what page src[i] held, for all i at once."""
    new = pool.copy()
    for s, d in zip(src, dst):
        new[:, d] = pool[:, s]
    return new


def compact(tables, num_pages):
    """(src, dst, new tables, live pages) of moving the named pages to the ids below their number."""
    live = sorted({int(p) for t in tables for p in t})
    n = len(live)
    high = [p for p in live if p >= n]
    holes = [p for p in range(n) if p not in set(live)]
    to = dict(zip(high, holes))
    return high, holes, [np.array([to.get(int(p), int(p)) for p in t], dtype=np.int32) for t in tables], n
