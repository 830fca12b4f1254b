"""The launch rule of the attentions over pages (csrc/attn_paged.cu), restated: which way a batch's tiles are shared."""
import math

CTAS = 152


def row_tile(latent: int, group: int, hint: int) -> int:
    """Query rows of a row tile."""
    rows = hint * group
    return 16 if rows <= 16 else 32 if rows <= 32 else 64 if latent else 128


def together(p, latent: int) -> int:
    """Row tiles of the same keys that CTAs walk together."""
    group = p.num_q_heads // (1 if latent else p.num_kv_heads)
    n = row_tile(latent, group, p.max_new_tokens)
    if n < 128:
        return 1
    most = -(-p.max_new_tokens * group // n)
    return -(-most // -(-most // 8)) if p.total_tokens * group > p.num_reqs * (most - 1) * n else 1


def path(p, latent: int) -> str:
    """'whole', 'cluster 2' to 'cluster 8', or 'list' with its join: 'by item, wide', 'by item', 'by cta'."""
    heads = 1 if latent else p.num_kv_heads
    group = p.num_q_heads // heads
    n = row_tile(latent, group, p.max_new_tokens)
    items = heads * (p.total_tokens * group // n + p.num_reqs)
    tiles = -(-p.max_seqlen // 128)
    best, name = items * (tiles + 1) / CTAS + (2.5 if latent else 5), "list"
    whole = math.ceil(items / CTAS) * (tiles + 1)
    if whole <= best:
        best, name = whole, "whole"
    for c in (2, 4, 8):
        if items * c <= CTAS and math.ceil(tiles / c) + 1 < best:
            best, name = math.ceil(tiles / c) + 1, f"cluster {c}"
    if name != "list":
        return name
    joins = heads * (p.total_tokens * group // n + p.num_reqs * together(p, latent))
    return "list, by cta" if joins > CTAS else "list, by item, wide" if joins <= 16 else "list, by item"
