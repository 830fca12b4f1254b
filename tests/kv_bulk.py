"""tests/kv_reference.py's packing and unpacking of 4-bit caches for many tokens at once (compared with it slot by slot in
tests/test_kv_bulk.py), and cases built with them."""
from __future__ import annotations

import numpy as np
import torch

from block_sparse_long_gb300 import kv as C
from tests import kv_reference as ref
from tests.kv_helpers import table


def _nibbles(d: int, word: int) -> np.ndarray:
    """Value that each nibble of a row of codes has, for words of `word` values."""
    G = d // ref.GROUP
    j = np.arange(d)
    g, r = j // ref.GROUP, j % ref.GROUP
    at = np.empty(d, np.int64)
    at[((r // word) * G + g) * word + r % word] = j
    return at


def _rows(pages: int, H: int, P: int, d: int, phys, row, at, size):
    """Index of `size` bytes from byte `at` [N] of the tiles of tokens (phys [N], row [N]), all heads: [N, H, size]."""
    return (np.asarray(phys)[:, None, None], np.arange(H)[None, :, None], (np.asarray(row) // 16)[:, None, None],
            (np.asarray(at)[:, None] + np.arange(size))[:, None, :])


def _pieces(d: int, row):
    """(codes' first byte, scales' first byte) of K and of V in the tile, per token."""
    G, t = d // ref.GROUP, np.asarray(row) % 16
    yield t * (d // 2), 16 * d + t * 2 * G, 8
    yield 8 * d + ((t % 2) * 8 + t // 2) * (d // 2), 16 * d + 32 * G + t * 2 * G, 4


def put(cache: np.ndarray, phys, row, k: np.ndarray, v: np.ndarray) -> None:
    """Tokens' keys and values [N, H, d] (bf16 values) into rows `row` of pages `phys`; cache uint8 [pages, H, P, 9 d / 8]."""
    pages, H, P, _ = cache.shape
    d = k.shape[-1]
    tiles = cache.reshape(pages, H, P // 16, 18 * d)
    for (codes_at, scales_at, word), x in zip(_pieces(d, row), (k, v)):
        c, s = ref.quantise(x)
        order = _nibbles(d, word)
        nib = np.abs(c)[..., order].astype(np.uint8) | ((c < 0)[..., order[np.arange(d) ^ 2]].astype(np.uint8) << 3)
        tiles[_rows(pages, H, P, d, phys, row, codes_at, d // 2)] = nib[..., 0::2] | (nib[..., 1::2] << 4)
        bits = (s.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        tiles[_rows(pages, H, P, d, phys, row, scales_at, d // 16)] = bits.view(np.uint8)


def get(cache: np.ndarray, phys, row, d: int):
    """float64 keys and values [N, H, d] of rows `row` of pages `phys`."""
    pages, H, P, _ = cache.shape
    tiles = cache.reshape(pages, H, P // 16, 18 * d)
    out = []
    for codes_at, scales_at, word in _pieces(d, row):
        b = tiles[_rows(pages, H, P, d, phys, row, codes_at, d // 2)]
        nib = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], d)
        c = (nib & 7) * np.where(nib[..., np.arange(d) ^ 2] & 8, -1.0, 1.0)
        x = np.empty_like(c)
        x[..., _nibbles(d, word)] = c
        s = np.ascontiguousarray(tiles[_rows(pages, H, P, d, phys, row, scales_at, d // 16)]).view(np.uint16).astype(np.uint32) << 16
        out.append(x * np.repeat(s.view(np.float32).astype(np.float64), ref.GROUP, -1))
    return out


def packed(rng, lens, heads, P, d, missing=(), edit=None):
    """As kv_helpers.packed: (cache on the GPU, table, k, v), for long requests."""
    pages = max(1, max(-(-n // P) for n in lens))
    total = len(lens) * pages + 3
    t = table(rng, len(lens), pages, total, missing)
    cache = rng.integers(0, 256, C.kv4_cache_shape(total, heads, P, d), dtype=np.uint8)
    ks, vs = [], []
    for b, n in enumerate(lens):
        k, v = (ref.bf16(rng.standard_normal((n, heads, d)) * f) for f in (1.0, 0.7))
        if edit is not None:
            edit(b, k, v)
        phys = t[b, np.arange(n) // P].astype(np.int64)
        there = (phys >= 0) & (phys < total)
        put(cache, phys[there], (np.arange(n) % P)[there], k[there], v[there])
        ks.append(ref.rounded(k))
        vs.append(ref.rounded(v))
    return torch.from_numpy(cache).to("cuda"), t, ks, vs
