"""Plain float64 implementations of the calls of include/cosa_attn.h, for the tests: numpy, request by request, written from the
header's definitions.  bf16 arrays are float64 arrays of bf16 values."""
from __future__ import annotations

import numpy as np


def seen_of(length: int, new: int, masks=None) -> np.ndarray:
    """[new, length]: which slots each of the newest tokens sees; masks: one int per token, or None for a chain."""
    seen = np.ones((new, length), dtype=bool)
    for i in range(new):
        for j in range(new):
            seen[i, length - new + j] = j <= i if masks is None else bool(masks[i] >> j & 1)
    return seen


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, seen: np.ndarray, scale: float):
    """q [n, Hq, dk], k [L, Hkv, dk], v [L, Hkv, dv], seen [n, L] -> (out [n, Hq, dv], lse [n, Hq], sum of p |v|, the bound on
    the logits' error [n, Hq]).

    Bound: the fp32 accumulation of a matrix unit may truncate, 2^-23 of the magnitudes' sum for each of dk / 16 steps, after
    cutting 16 products to the width of the largest, 16 2^-24; the scaling and the exponent's argument are rounded in
    fp32, 4 2^-24 of the largest logit."""
    n, Hq, dk = q.shape
    L, Hkv, dv = v.shape
    g = Hq // Hkv
    out, lse, mag, err = np.zeros((n, Hq, dv)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, dv)), np.zeros((n, Hq))
    for i in range(n):
        at = np.nonzero(seen[i])[0]
        if not len(at):
            continue
        for h in range(Hq):
            kk, vv = k[at, h // g], v[at, h // g]
            with np.errstate(invalid="ignore", over="ignore"):
                x = kk @ q[i, h] * scale
                top = x.max()
                p = np.exp(x - top)
                lse[i, h] = top + np.log(p.sum())
                p /= p.sum()
                out[i, h], mag[i, h] = p @ vv, p @ np.abs(vv)
                size = np.abs(kk) @ np.abs(q[i, h]) * scale
            err[i, h] = (size.max() * (dk / 8 + 16) + np.abs(x).max() * 4) * 2.0 ** -24
    return out, lse, mag, err


def rotate(x: np.ndarray, pos: np.ndarray, inv_freq: np.ndarray, interleaved: bool):
    """[T, H, 64] -> (result, |a| + |b| of the values each was formed from)."""
    y, mag = x.copy(), np.abs(x)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = (pos.astype(np.float64) * inv_freq[i])[:, None]
        y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
        y[..., b] = x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def norm(c: np.ndarray, w, eps: float) -> np.ndarray:
    if w is None:
        return c
    with np.errstate(invalid="ignore"):
        return c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * w


def commit(rows: np.ndarray, there: np.ndarray, length: int, new: int, path) -> np.ndarray:
    """rows [slots, ...] of one request after the rows of path moved behind the context; there: which slots have a page."""
    out, base = rows.copy(), length - new
    for i, j in enumerate(path):
        if there[base + i] and there[base + j]:
            out[base + i] = rows[base + j]
    return out
