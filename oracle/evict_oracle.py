"""fp64 oracle of differential attention, weighing and eviction (include/kamera_step.h).

NumPy only, from the definitions; no code shared with the library. Functions that compute also return what the
tests' error bounds are made of.
"""
import numpy as np

from oracle import step_oracle as so


def lam(vectors, init):
    """lambda from its four vectors (None: the constant), and the sum of the absolute terms that its rounding goes by."""
    if vectors is None:
        return init, abs(init)
    q1, k1, q2, k2 = np.asarray(vectors, np.float64)
    a, b = np.exp(q1 @ k1), np.exp(q2 @ k2)
    return a - b + init, a * (1 + np.abs(q1 * k1).sum()) + b * (1 + np.abs(q2 * k2).sum()) + abs(init)


def combine(first, second, value):
    """first - lambda * second over the maps' results [..., 2 d]."""
    return first - value * second


def head_norm(x, weight, eps, scale):
    """x / sqrt(mean(x^2) + eps) * weight * scale over the last axis; zeros stay zeros."""
    n = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return np.where(n == 0, 0.0, x / np.where(n == 0, 1.0, n)) * weight * scale


def weights(q, keys, lse, scale, last):
    """What queries [n][G][dk] (statistics lse [n][G]) give keys [T][dk], query i seeing keys 0..last[i].
    Returns (sums [T], sums of weight * (absolute score terms, |score| and |lse|))."""
    total, terms = np.zeros(keys.shape[0]), np.zeros(keys.shape[0])
    for i in range(q.shape[0]):
        t = int(last[i]) + 1
        if t <= 0:
            continue
        for g in range(q.shape[1]):
            if np.isneginf(lse[i, g]):
                continue
            s = scale * (keys[:t] @ q[i, g])
            p = np.exp(s - lse[i, g])
            total[:t] += p
            terms[:t] += p * (abs(scale) * (np.abs(keys[:t]) @ np.abs(q[i, g])) + np.abs(s) + abs(lse[i, g]))
    return total, terms


def stays(scores, keep, first, last):
    """Tokens that stay of a sequence with group scores [n] (already summed): ascending numbers."""
    n = len(scores)
    if keep >= n:
        return np.arange(n)
    key = np.where(np.isnan(scores), -np.inf, scores.astype(np.float64))
    nan = np.isnan(scores)
    middle = sorted(range(first, n - last), key=lambda t: (nan[t], -key[t], t))
    return np.array(sorted(list(range(first)) + middle[:keep - first - last] + list(range(n - last, n))), dtype=np.int64)


def group_scores(scores):
    """fp32 sum of a group's heads' scores [heads][n], one head after the other."""
    x = scores[0].astype(np.float32)
    for y in scores[1:]:
        x = x + y.astype(np.float32)
    return x


def turned(rows, back, base, band0, gptj=False):
    """rows [n][d] whose columns from band0 on turn back by `back` [n] positions. (result, sums of |terms|)."""
    phi = so.phases(-np.asarray(back, np.float64), rows.shape[1] - band0, base)
    y, t = so.rotate(rows[:, band0:], phi, gptj)
    return np.concatenate([rows[:, :band0], y], 1), np.concatenate([np.zeros((rows.shape[0], band0)), t], 1)
