"""The operators of a prompt that arrives in chunks, from their definitions, in float64 on the CPU."""
from __future__ import annotations

import numpy as np

from .attention import masked_rows


def norm_rope_rows(x, weight, eps, positions, inv_freq, interleaved: bool) -> np.ndarray:
    """x [tokens, heads, D]: each row normalized (weight not None), its first 2 len(inv_freq) dims turned."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = 0 if inv_freq is None else len(inv_freq)
    if not half:
        return y
    # (float64 holds position * frequency to 2^-53, far below what a test asks)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    first, second = rope_pairs(half, interleaved)
    a, b = y[..., first], y[..., second]
    out = y.copy()
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    return out


def rope_pairs(half: int, interleaved: bool):
    """The dims of the first and of the second member of every pair."""
    j = np.arange(half)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + half)


def chunk_sees(n: int, length: int, window: int = 0) -> np.ndarray:
    """bool [n, length]: row i, at position length - n + i, sees keys 0 .. that position, the last `window` of them."""
    row, key = np.arange(length - n, length)[:, None], np.arange(length)
    sees = key <= row
    return sees & (key > row - window) if window else sees


def chunk_rows(q, k, v, window: int, sm_scale: float):
    """q [n, Hq, D] behind its context in k, v [T, Hkv, D]: out [n, Hq, D] and the log-sum-exp [n, Hq], float64."""
    sees = chunk_sees(len(q), len(k), window)
    out = masked_rows(q, k, v, sees, sm_scale)
    return out, logits_lse(logits(q, k, sees, sm_scale))


def logits(q, k, sees, sm_scale: float) -> np.ndarray:
    """[Hq, n, T] scaled scores, -inf where a row does not see the key."""
    q, k = np.asarray(q, np.float64), np.asarray(k, np.float64)
    group = q.shape[1] // k.shape[1]
    s = np.stack([q[:, h] @ k[:, h // group].T for h in range(q.shape[1])]) * sm_scale
    return np.where(sees, s, -np.inf)


def logits_lse(s) -> np.ndarray:
    """[n, Hq] log of the sum of the exponentials; -inf for rows that see nothing."""
    top = s.max(-1, keepdims=True, initial=-np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    with np.errstate(divide="ignore"):
        return (np.log(np.exp(s - safe).sum(-1)) + safe[..., 0]).T


def key_weights(q, k, lse, sm_scale: float) -> np.ndarray:
    """[Hkv, T]: the sum over rows and a group's heads of exp(score - lse), for a chunk at the end of its keys."""
    s = logits(q, k, chunk_sees(len(q), len(k)), sm_scale)
    p = np.exp(s - np.asarray(lse, np.float64).T[..., None])
    return p.reshape(k.shape[1], -1, len(k)).sum(1)


def kept_tokens(weights, n: int, sink: int, recent: int) -> np.ndarray:
    """The n tokens of len(weights) that an eviction keeps, in order (NaN weighs least)."""
    T = len(weights)
    n = min(n, T)
    recent = min(recent, n)
    sink = min(sink, n - recent)
    order = []
    for i in range(sink, T - recent):
        w = float(weights[i])
        order.append((w != w, -w if w == w else 0.0, i))
    order.sort()
    return np.array(sorted(list(range(sink)) + [i for _, _, i in order[:n - sink - recent]] +
                           list(range(T - recent, T))), np.int64)
