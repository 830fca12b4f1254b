"""Plain float64 / integer implementations of the calls of include/cosa_kv.h, for the tests: numpy loops over requests,
written from the header's definitions.  bf16 arrays are float64 arrays of bf16 values."""
from __future__ import annotations

import math

import numpy as np
import torch

GROUP, TILE = 32, 16


def bf16(x) -> np.ndarray:
    """float64 -> the nearest bf16 values (ties to even), as float64; each from its own bits."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)                                   # x = m 2^e, 0.5 <= |m| < 1
    step = np.exp2(np.maximum(e - 8, -133).astype(np.float64))
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(np.isfinite(x), np.rint(x / step) * step, x)
        return np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, y), y)


def to_f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def quantise(x: np.ndarray):
    """[..., d] -> (codes [..., d] in -7..7, scales [..., d / 32]); a group that is not finite has a NaN scale."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    bad = ~np.isfinite(g).all(-1)
    amax = np.abs(np.where(bad[..., None], 0.0, g)).max(-1)
    s = bf16(amax / 7)
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.clip(np.rint(np.where(s[..., None] > 0, g / np.where(s > 0, s, 1)[..., None], 0.0)), -7, 7)
    c = np.where(bad[..., None], 0.0, c).reshape(x.shape)
    return c, np.where(bad, np.nan, s)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return codes * np.repeat(scales, GROUP, -1)


def rounded(x: np.ndarray) -> np.ndarray:
    """What a 4-bit store of x stands for."""
    return values(*quantise(x))


def unpack_slot(cache: np.ndarray, phys: int, h: int, row: int, d: int):
    """float64 (key [d], value [d]) of row `row` of a page, from a uint8 cache [pages, Hkv, P, 9 d / 8]."""
    G = d // GROUP
    page = cache[phys, h].reshape(-1)
    tile = page[(row // TILE) * 18 * d:(row // TILE + 1) * 18 * d]
    t = row % TILE
    out = []
    for which, at in ((0, t), (1, (t % 2) * 8 + t // 2)):
        codes = tile[which * 8 * d + at * (d // 2):which * 8 * d + (at + 1) * (d // 2)]
        nib = np.empty(d, np.int64)
        nib[0::2], nib[1::2] = codes & 15, codes >> 4
        word = 8 if which == 0 else 4
        x = np.empty(d)
        for j in range(d):
            g, r = j // GROUP, j % GROUP
            n = ((r // word) * G + g) * word + r % word
            x[j] = (nib[n] & 7) * (-1.0 if nib[n ^ 2] & 8 else 1.0)
        sc = tile[16 * d + which * 2 * TILE * G + t * 2 * G:][:2 * G].copy().view(np.uint16).astype(np.uint32) << 16
        out.append(x * np.repeat(sc.view(np.float32).astype(np.float64), GROUP))
    return out


def unpack_request(cache: np.ndarray, table: np.ndarray, n: int, d: int):
    """float64 keys and values [n, Hkv, d] of slots 0 .. n - 1, and whether each slot exists."""
    pages, H, P, _ = cache.shape
    k, v, there = np.zeros((n, H, d)), np.zeros((n, H, d)), np.zeros(n, bool)
    for s in range(n):
        phys = int(table[s // P])
        if 0 <= phys < pages:
            there[s] = True
            for h in range(H):
                k[s, h], v[s, h] = unpack_slot(cache, phys, h, s % P, d)
    return k, v, there


def pack_slot(cache: np.ndarray, phys: int, h: int, row: int, key: np.ndarray, value: np.ndarray) -> None:
    """Store one token's key and value (bf16 values) of one head."""
    d = key.shape[0]
    G = d // GROUP
    page = cache[phys, h].reshape(-1)
    tile = page[(row // TILE) * 18 * d:(row // TILE + 1) * 18 * d]
    t = row % TILE
    for which, at, x in ((0, t, key), (1, (t % 2) * 8 + t // 2, value)):
        c, s = quantise(x)
        word = 8 if which == 0 else 4
        nib = np.zeros(d, np.uint8)
        for j in range(d):
            g, r = j // GROUP, j % GROUP
            n = ((r // word) * G + g) * word + r % word
            nib[n] |= int(abs(c[j]))
            nib[n ^ 2] |= 8 if c[j] < 0 else 0
        tile[which * 8 * d + at * (d // 2):which * 8 * d + (at + 1) * (d // 2)] = nib[0::2] | (nib[1::2] << 4)
        bits = (s.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        tile[16 * d + which * 2 * TILE * G + t * 2 * G:][:2 * G] = bits.view(np.uint8)


def norm_rope(x: np.ndarray, w, pos: np.ndarray, inv_freq: np.ndarray, interleaved: bool, eps: float):
    """[T, H, d] -> (result, magnitude): the result in float64, and |a| + |b| of the values it was formed from."""
    x = x.astype(np.float64)
    if w is not None:
        with np.errstate(invalid="ignore"):
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y, mag = x.copy(), np.abs(x)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = (pos.astype(np.float64) * inv_freq[i])[:, None]
        y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
        y[..., b] = x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, there: np.ndarray, scale: float):
    """One request: q [n, Hq, d], k and v [L, Hkv, d] -> (out, sum of p |v|, p [n, Hq, L])."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    g = Hq // Hkv
    out, mag, p = np.zeros((n, Hq, d)), np.zeros((n, Hq, d)), np.zeros((n, Hq, L))
    for i in range(n):
        seen = there & (np.arange(L) < L - n + i + 1)
        idx = np.nonzero(seen)[0]
        if not len(idx):
            continue
        for h in range(Hq):
            s = (k[idx, h // g] @ q[i, h]) * scale
            with np.errstate(invalid="ignore"):
                e = np.exp(s - s.max())
                p[i, h, idx] = e / e.sum()
                out[i, h] = p[i, h, idx] @ v[idx, h // g]
                mag[i, h] = p[i, h, idx] @ np.abs(v[idx, h // g])
    return out, mag, p


def logit_error(q: np.ndarray, k: np.ndarray, scale: float) -> float:
    """Bound on the error of any logit of the request: its sum runs in fp32 on a matrix unit that truncates, 48 2^-24 of the
    sum of the magnitudes (16-term groups aligned to their largest term and cut to fp32 width, added to a truncating sum);
    the terms are q times a code of at most 7, times the group's scale."""
    if not k.size or not q.size:
        return 0.0
    amax = np.nanmax(np.where(np.isfinite(k), np.abs(k), 0.0).reshape(-1, k.shape[-1] // GROUP, GROUP), axis=(0, 2)) / 7
    qs = np.abs(q).reshape(-1, q.shape[-1] // GROUP, GROUP).sum(-1)
    return float((qs * amax).sum(-1).max() * 7 * 48 * 2.0 ** -24 * scale)


def evict(weights: np.ndarray, there: np.ndarray, budget: int, sink: int, recent: int) -> np.ndarray:
    """Kept slots, ascending, of one (request, kv head): weights [L] float32, there [L]."""
    L = len(weights)

    def order(s):
        forced = s < sink or s >= L - recent
        w = float(weights[s])
        return (not forced, math.isnan(w), -w if not math.isnan(w) else 0.0, s)

    slots = sorted((s for s in range(L) if there[s]), key=order)
    return np.array(sorted(slots[:budget]), dtype=np.int64)
