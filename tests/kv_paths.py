"""Which way cosa_kv4_attention shares its work: the launch rule of kv_attention.cu restated, so that a test can say which of its
kernels it reaches."""
from __future__ import annotations

import numpy as np
import torch

SMS = 152


def row_groups(p) -> int:
    """Eights of query rows of a row tile."""
    rows = min(p.max_new_tokens, p.total_tokens) * (p.num_q_heads // p.num_kv_heads)
    return 1 if rows <= 8 else 3 if 16 < rows <= 24 else 2


def items(p) -> int:
    """(request, kv head, row tile), as far as the parameters tell."""
    rows = min(p.max_new_tokens, p.total_tokens) * (p.num_q_heads // p.num_kv_heads)
    return p.num_reqs * p.num_kv_heads * -(-rows // (8 * row_groups(p)))


def shares_a_list(p) -> bool:
    """Whether the batch is shared as one list and joined by a second kernel; else clusters have an item each."""
    nt, n = row_groups(p), items(p)
    unit = 32 if nt <= 2 else 16
    resident = SMS * (3 if nt == 1 else 2)
    units, ctas = -(-p.max_seqlen // unit), 1
    while ctas < 16 and 2 * ctas * n <= resident and ctas * 4 < units:
        ctas *= 2
    tokens = -(-units // (ctas * 4)) * unit
    return not (ctas * n <= resident and tokens <= (512 if 2 * ctas * n >= resident else 256))


def parts_of_the_longest(p, lens) -> int:
    """CTAs that share the longest request's first item in a list, at least (equal shares of the items' units, each item with 12
    more than its own; a CTA has four units or more)."""
    nt = row_groups(p)
    unit, resident = (32 if nt <= 2 else 16), SMS * (3 if nt == 1 else 2)
    own = [max(1, -(-n // unit)) for n in lens]
    total = sum(u + 12 for u in own) * p.num_kv_heads
    each = -(-total // max(1, min(resident, total // 4)))
    return max(own) // each


def widened(c, tokens=40000):
    """A case of tests/test_gpu_kv.py's attend() with page tables for `tokens`, more than any cluster takes."""
    p, P = c["p"], c["P"]
    pages = -(-tokens // P)
    t = np.full((p.num_reqs, pages), -1, np.int32)
    t[:, :c["t"].shape[1]] = c["t"]
    if c["acc"] is not None:
        acc = torch.rand(p.num_reqs, p.num_kv_heads, pages * P, device=c["acc"].device)
        acc[..., :c["acc"].shape[2]] = c["acc"]
        c["acc"] = acc
    c["t"], p.max_seqlen, p.max_pages_per_req = t, pages * P, pages
    assert shares_a_list(p)
    return c
