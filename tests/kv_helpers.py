"""Inputs shared by the tests of include/cosa_kv.h's calls."""
from __future__ import annotations

import numpy as np
import torch

from block_sparse_long_gb300 import kv as C
from tests import kv_reference as ref

DEV = "cuda"


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def cu_of(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]))


def bf(rng, *shape, scale=1.0):
    """Random bf16 values: a CUDA tensor."""
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * scale).to(torch.bfloat16).to(DEV)


def table(rng, reqs, pages, total, missing=()):
    """A shuffled page table; entries (b, page) of `missing` point nowhere."""
    t = rng.permutation(total)[: reqs * pages].reshape(reqs, pages).astype(np.int32)
    for n, (b, p) in enumerate(missing):
        t[b, p] = -1 if n % 2 == 0 else total + n
    return t


def noise_cache(rng, pages, heads, P, d):
    """A cache full of arbitrary bytes (NaN scales among them)."""
    return torch.from_numpy(rng.integers(0, 256, C.kv4_cache_shape(pages, heads, P, d), dtype=np.uint8)).to(DEV)


def packed(rng, lens, heads, P, d, pages_per_req=None, missing=(), edit=None):
    """(cache, table, k, v): requests of random keys and values packed by the reference into noise; k[b], v[b] are what
    the cache stands for, [L, heads, d]."""
    pages = pages_per_req or max(1, max(-(-n // P) for n in lens))
    total = len(lens) * pages + 3
    t = table(rng, len(lens), pages, total, missing)
    cache = rng.integers(0, 256, C.kv4_cache_shape(total, heads, P, d), dtype=np.uint8)
    ks, vs = [], []
    for b, n in enumerate(lens):
        k, v = (ref.bf16(rng.standard_normal((n, heads, d)) * f) for f in (1.0, 0.7))
        if edit is not None:
            edit(b, k, v)
        for s in range(n):
            phys = int(t[b, s // P])
            if 0 <= phys < total:
                for h in range(heads):
                    ref.pack_slot(cache, phys, h, s % P, k[s, h], v[s, h])
        ks.append(ref.rounded(k))
        vs.append(ref.rounded(v))
    return torch.from_numpy(cache).to(DEV), t, ks, vs


def exists(t, b, n, P, total):
    e = t[b].astype(np.int64)
    ok = (e >= 0) & (e < total)
    return np.array([ok[s // P] for s in range(n)], dtype=bool)


def new_status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def ok(status):
    torch.cuda.synchronize()
    assert int(status.item()) == 0, int(status.item())
