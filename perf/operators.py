"""The operators around the sparse prefill, each in its plain form and as the library's call.

  rope    norms of queries and keys per head with the position rotation, K and V into bf16 pages or K into rows
  store   K and V rounded to 4 bits (groups of 32 along the head, one bf16 scale each), from rows or from bf16 pages;
          the stored values are read back with the load call, since a cache is compared by the values it stands for
  load    a 4-bit cache back into bf16 pages
  attn    attention of one to a few new tokens per request over the 4-bit cache, optionally adding the
          attention weight that each slot received to an accumulator
  evict   the slots with the largest accumulated weights (and the first and last ones) moved in order into other pages;
          the destination is read back with the load call

`own` chooses between the plain form (torch operations in 32 bits) and the library.
"""
import math
import random

import torch

own = False

GROUP = 32  # values that share a scale
DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _lens(c):
    """Request lengths of a case: the first is the longest, the others spread between the bounds."""
    r = random.Random(c["len_seed"])
    return [c["max_len"]] + [r.randint(c["min_len"], c["max_len"]) for _ in range(c["reqs"] - 1)]


def listed():
    gqa = dict(q_heads=32, kv_heads=8, d=128, page=64)
    return [
        # a decode step of 64 requests: one new token each, keys to rows for the 4-bit append
        dict(name="rope decode 64", op="rope", reqs=64, min_len=1, max_len=1, ctx=8000, len_seed=1, rot=128,
             interleaved=False, to="rows", norm=True, **gqa),
        # a ragged chunk of five prompts, half of each head rotated in interleaved pairs, into 16-token pages
        dict(name="rope ragged 5 partial", op="rope", reqs=5, min_len=37, max_len=2011, ctx=1001, len_seed=2, q_heads=12,
             kv_heads=4, d=64, page=16, rot=32, interleaved=True, to="pages", norm=True),
        # the 128K-token prompt of the benchmark workload: q rows and bf16 pages as the sparse prefill reads them
        dict(name="rope prefill 128k", op="rope", reqs=1, min_len=131072, max_len=131072, ctx=0, len_seed=3, rot=128,
             interleaved=False, to="pages", norm=True, **gqa),
        # the decode step's append: 64 requests, one token each
        dict(name="store append 64", op="store", form="rows", reqs=64, min_len=1, max_len=1, ctx=4000, len_seed=4, **gqa),
        # a 32K-token prompt's bf16 pages to 4 bits after its prefill
        dict(name="store pages 32k", op="store", form="pages", reqs=1, min_len=32768, max_len=32768, ctx=0, len_seed=5, **gqa),
        # a short conversation's cache back to bf16, heads of 64
        dict(name="load 2k d64", op="load", reqs=1, min_len=2048, max_len=2048, ctx=0, len_seed=6, q_heads=1, kv_heads=1, d=64, page=64),
        # ragged contexts (16K to 128K) handed back to the sparse prefill, the later part of each only
        dict(name="load ragged 4", op="load", reqs=4, min_len=16384, max_len=131072, ctx=5003, len_seed=7, **gqa),
        # decode of one short prompt: latency
        dict(name="attn 1x777", op="attn", reqs=1, min_len=777, max_len=777, new=1, len_seed=8, weights=False, **gqa),
        # decode of one 128K-token context: the cache is read by the whole card
        dict(name="attn 1x128k", op="attn", reqs=1, min_len=131072, max_len=131072, new=1, len_seed=9, weights=False, **gqa),
        # a serving batch, two tokens per request (a drafted one), adding up the weights for eviction
        dict(name="attn 48 ragged weights", op="attn", reqs=48, min_len=1000, max_len=16384, new=2, len_seed=10, weights=True, **gqa),
        # one 128K context thinned to an eighth
        dict(name="evict 1x128k", op="evict", reqs=1, min_len=131072, max_len=131072, len_seed=11, budget=16384, sink=4,
             recent=512, **gqa),
        # a ragged batch thinned to 2000 slots (some are shorter and only move)
        dict(name="evict 24 ragged", op="evict", reqs=24, min_len=300, max_len=9000, len_seed=12, budget=2000, sink=16,
             recent=200, **gqa),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice((64, 128))
    kv = rng.choice((1, 2, 4, 8))
    c = dict(q_heads=kv * rng.choice((1, 2, 3, 4, 7, 8)), kv_heads=kv, d=d, page=rng.choice((16, 32, 64, 128)),
             len_seed=rng.randrange(1 << 30))
    op = rng.choice(("rope", "store", "load", "attn", "attn", "evict"))
    reqs = _log(rng, 1, 64)
    # tokens of the whole batch at most: below the largest listed case of the operator
    most = ((1 << 16) if op == "rope" else (1 << 17)) // reqs
    top = _log(rng, 1, most)
    c.update(op=op, reqs=reqs, max_len=top, min_len=rng.randint(1, top))
    if op == "rope":
        c.update(ctx=rng.randint(0, 2000), rot=rng.choice((d, d, d // 2, 16)), interleaved=rng.random() < 0.3,
                 to=rng.choice(("pages", "rows")), norm=rng.random() < 0.8)
    elif op == "store":
        c.update(form=rng.choice(("rows", "pages")), ctx=rng.randint(0, 1000))
    elif op == "load":
        c.update(ctx=rng.randint(0, top // 2))
    elif op == "attn":
        c.update(new=rng.choice((1, 1, 1, 2, 3, 5)), weights=rng.random() < 0.4)
    else:
        budget = _log(rng, 1, max(2, top // 2))
        sink = rng.randint(0, min(8, budget))
        c.update(budget=budget, sink=sink, recent=rng.randint(0, budget - sink))
    return c


def _slots(c):
    """(first, end) of the slots that a store or load of the case covers, per request."""
    lens = _lens(c)
    if c["op"] == "load":
        return [(min(c["ctx"], n), n) for n in lens]
    return [(c["ctx"], c["ctx"] + n) for n in lens]


def work(c):
    Hq, Hkv, d = c["q_heads"], c["kv_heads"], c["d"]
    packed = 2 * (d // 2 + d // GROUP * 2) * Hkv      # bytes of a token's K and V in 4 bits
    full = 2 * d * 2 * Hkv                            # and in bf16
    lens = _lens(c)
    n = sum(lens)
    if c["op"] == "rope":
        rows = Hq + Hkv + (Hkv if c["to"] == "pages" else 0)
        return {"bytes": 2 * n * rows * d * 2, "flops": 10 * n * (Hq + Hkv) * d}
    if c["op"] == "store":
        return {"bytes": n * (full + packed) * 2, "flops": 4 * n * Hkv * d * 2}
    if c["op"] == "load":
        n = sum(e - s for s, e in _slots(c))
        return {"bytes": max(1, n * (full + packed)), "flops": n * Hkv * d * 2}
    if c["op"] == "attn":
        q = c["reqs"] * c["new"] * Hq * d * 2 * 2
        return {"bytes": n * packed + q + (8 * n * Hkv if c["weights"] else 0), "flops": 4 * n * c["new"] * Hq * d}
    kept = sum(min(v, c["budget"]) for v in lens)
    # weights in, kept rows in and out, weights and indices out; then the read-back
    return {"bytes": 4 * n * Hkv + 2 * kept * packed + 4 * n * Hkv + 4 * kept * Hkv + kept * (packed + full),
            "flops": 4 * n * Hkv}


# ---------------------------------------------------------------------------------------------------------------
# the 4-bit layout, in torch: pages of 16-token tiles, per (page, kv head, tile) the bytes
#   K codes [16][d/2], V codes [16][d/2], K scales bf16 [16][d/32], V scales bf16 [16][d/32]
# a K row's 32-bit word c*G+g holds values 32g+8c.. (8 codes), a V row's 16-bit word i*G+g values 32g+4i.. (4 codes),
# G = d/32, low nibble first; the V row of token t of its tile is row (t%2)*8 + t//2; in each group of four nibbles, nibble n
# has the magnitude of code n in its three low bits and the sign of code n ^ 2 in its high bit
# ---------------------------------------------------------------------------------------------------------------
def _nibbles_to_bytes(u):
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _bytes_to_nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _other_sign(x):
    """Entries n ^ 2 of each four."""
    return x.unflatten(-1, (-1, 2, 2)).flip(-2).flatten(-3)


def _codes_to_nibbles(c):
    """Codes in -7 .. 7, in the order of the layout's words."""
    return c.abs().to(torch.uint8) | (_other_sign(c < 0).to(torch.uint8) << 3)


def _nibbles_to_codes(u):
    c = (u & 7).float()
    return torch.where(_other_sign(u) > 7, -c, c)


def _quantise(x):
    """fp32 [..., d] -> (codes in fp32 [..., d], scales bf16 [..., d/32])."""
    g = x.unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1) / 7).to(torch.bfloat16)
    sf = s.float().unsqueeze(-1)
    code = torch.where(sf > 0, (g / sf).round().clamp(-7, 7), torch.zeros_like(g))
    return code.flatten(-2), s


def _pack(k, v):
    """fp32 K, V [pages, P, H, d] -> uint8 [pages, H, P, 9d/8]."""
    np_, P, H, d = k.shape
    G, nt = d // GROUP, P // 16
    out = []
    for x, inner in ((k, (G, 4, 8)), (v, (G, 8, 4))):
        u, s = _quantise(x)
        u = u.permute(0, 2, 1, 3).reshape(np_, H, nt, 16, *inner).transpose(-3, -2).reshape(np_, H, nt, 16, d)
        s = s.permute(0, 2, 1, 3).reshape(np_, H, nt, 16 * G).contiguous().view(torch.uint8)
        out.append((_nibbles_to_bytes(_codes_to_nibbles(u)), s))
    (ku, ks), (vu, vs) = out
    vu = vu.unflatten(3, (8, 2)).transpose(3, 4).flatten(3, 4)
    return torch.cat((ku.flatten(3), vu.flatten(3), ks, vs), -1).reshape(np_, H, P, 9 * d // 8).contiguous()


def _unpack(rec, d):
    """uint8 [n, H, P, 9d/8] -> fp32 K, V [n, P, H, d]."""
    n, H, P, _ = rec.shape
    G, nt, half = d // GROUP, P // 16, 8 * d
    t = rec.reshape(n, H, nt, 18 * d)
    ku = t[..., :half].unflatten(-1, (16, d // 2))
    vu = t[..., half:2 * half].unflatten(-1, (2, 8, d // 2)).transpose(3, 4).flatten(3, 4)
    sc = t[..., 2 * half:].contiguous().view(torch.bfloat16).float().reshape(n, H, nt, 2, 16, G)
    got = []
    for j, (u, inner) in enumerate(((ku, (4, G, 8)), (vu, (8, G, 4)))):
        c = _nibbles_to_codes(_bytes_to_nibbles(u)).reshape(n, H, nt, 16, *inner).transpose(-3, -2)
        x = c.reshape(n, H, nt, 16, G, GROUP) * sc[:, :, :, j].unsqueeze(-1)
        got.append(x.reshape(n, H, P, d).transpose(1, 2))
    return got


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    return _i32([0] + [sum(lens[: i + 1]) for i in range(len(lens))])


def _table(g, reqs, pages, spare=0):
    """A shuffled page table [reqs, pages], and how many pages the cache has."""
    n = reqs * pages + spare
    return torch.randperm(n, generator=g, device=DEV)[: reqs * pages].to(torch.int32).reshape(reqs, pages), n


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _kv_values(g, pages, P, H, d):
    """Keys with a few large channels per head, as keys have, and plain values."""
    gain = torch.ones(H, d, device=DEV)
    gain.scatter_(1, torch.randint(0, d, (H, 4), generator=g, device=DEV), 4.0)
    k = _normal(g, pages, P, H, d).float() * gain
    return k, _normal(g, pages, P, H, d).float()


def _packed_cache(g, n, c):
    """A 4-bit cache of n pages, filled in parts to bound the memory."""
    P, H, d = c["page"], c["kv_heads"], c["d"]
    cache = torch.empty(n, H, P, 9 * d // 8, dtype=torch.uint8, device=DEV)
    part = max(1, (1 << 26) // (P * H * d))
    for at in range(0, n, part):
        k, v = _kv_values(g, min(part, n - at), P, H, d)
        cache[at:at + part] = _pack(k.to(torch.bfloat16).float(), v)
    return cache


def prepare(c, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    op, B, Hq, Hkv, d, P = c["op"], c["reqs"], c["q_heads"], c["kv_heads"], c["d"], c["page"]
    lens = _lens(c)
    s = dict(case=c, lens=lens, cu=_cu(lens))
    if op == "rope":
        T = sum(lens)
        qkv = _normal(g, T, (Hq + 2 * Hkv) * d)       # one row of the projection: queries, keys, values
        s["q"] = qkv[:, : Hq * d].unflatten(1, (Hq, d))
        s["k"] = qkv[:, Hq * d: (Hq + Hkv) * d].unflatten(1, (Hkv, d))
        s["v"] = qkv[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
        s["wq"] = (1 + 0.2 * _normal(g, d)) if c["norm"] else None
        s["wk"] = (1 + 0.2 * _normal(g, d)) if c["norm"] else None
        s["inv"] = 1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        start = [c["ctx"] + (7 * b) % 101 for b in range(B)]
        s["start"] = _i32(start)
        s["pos"] = torch.cat([torch.arange(f, f + n, device=DEV, dtype=torch.int32) for f, n in zip(start, lens)])
        s["q_out"] = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV)
        if c["to"] == "pages":
            pages = -(-max(f + n for f, n in zip(start, lens)) // P)
            s["pt"], n = _table(g, B, pages)
            s["k_cache"] = torch.zeros(n, P, Hkv, d, dtype=torch.bfloat16, device=DEV)
            s["v_cache"] = torch.zeros_like(s["k_cache"])
        else:
            s["k_out"] = torch.zeros(T, Hkv, d, dtype=torch.bfloat16, device=DEV)
    elif op in ("store", "load"):
        slots = _slots(c)
        pages = max(1, -(-max(e for _, e in slots) // P))
        s["pt"], n = _table(g, B, pages)               # the 4-bit pages
        s["pt16"], n16 = _table(g, B, pages)           # the bf16 pages
        s["start"], s["kv_len"] = _i32([a for a, _ in slots]), _i32([e for _, e in slots])
        s["slots"] = slots
        s["k_back"] = torch.zeros(n16, P, Hkv, d, dtype=torch.bfloat16, device=DEV)
        s["v_back"] = torch.zeros_like(s["k_back"])
        if op == "load":
            s["cache"] = _packed_cache(g, n, c)
        else:
            s["cache"] = torch.zeros(n, Hkv, P, 9 * d // 8, dtype=torch.uint8, device=DEV)
            if c["form"] == "rows":
                kv = _normal(g, sum(lens), 2 * Hkv * d)
                s["k"], s["v"] = kv[:, : Hkv * d].unflatten(1, (Hkv, d)), kv[:, Hkv * d:].unflatten(1, (Hkv, d))
            else:
                s["k16"], s["v16"] = (x.to(torch.bfloat16) for x in _kv_values(g, n16, P, Hkv, d))
    else:
        pages = -(-c["max_len"] // P)
        s["kv_len"] = _i32(lens)
        if op == "attn":
            s["pt"], n = _table(g, B, pages)
            s["cache"] = _packed_cache(g, n, c)
            new = [min(c["new"], v) for v in lens]
            s["cu_q"], s["new"] = _cu(new), new
            s["q"] = 1.5 * _normal(g, sum(new), Hq, d)
            s["out"] = torch.zeros_like(s["q"])
            # what earlier steps left in each slot: a few tens of steps' worth of weight
            s["acc"] = (-24 * torch.rand(B, Hkv, pages * P, generator=g, device=DEV).clamp_min(1e-6).log() / max(lens)
                        if c["weights"] else None)
        else:
            room = -(-c["budget"] // P)
            table, n = _table(g, B, pages + room)      # source pages, then pages of their own to move into
            s["pt"], s["dst"] = table[:, :pages].contiguous(), table[:, pages:].contiguous()
            s["cache"] = _packed_cache(g, n, c)
            s["acc"] = -torch.rand(B, Hkv, pages * P, generator=g, device=DEV).clamp_min(1e-6).log()
            s["pt16"], n16 = _table(g, B, room)
            s["k_back"] = torch.zeros(n16, P, Hkv, d, dtype=torch.bfloat16, device=DEV)
            s["v_back"] = torch.zeros_like(s["k_back"])
            s["new_len"] = torch.zeros(B, dtype=torch.int32, device=DEV)
            s["kept"] = torch.zeros(B, Hkv, c["budget"], dtype=torch.int32, device=DEV)
            s["acc_out"] = torch.zeros_like(s["acc"])
    if own:
        _plan(s)
    return s


def _plan(s):
    """The library's parameters and workspace, which a program makes once for its shapes."""
    from block_sparse_long_gb300 import kv as cosa

    c = s["case"]
    more = {}
    if c["op"] == "rope":
        more = dict(total_tokens=s["q"].shape[0], rotary_dim=c["rot"], interleaved=c["interleaved"])
        pages = s["pt"].shape[1] if "pt" in s else 1
        top = pages * c["page"]
        n16, n4 = (s["k_cache"].shape[0] if "k_cache" in s else 1), 1
    else:
        pages = s["pt"].shape[1]
        top = pages * c["page"]
        n16, n4 = (s["k_back"].shape[0] if "k_back" in s else 1), s["cache"].shape[0]
    if c["op"] == "store" and c["form"] == "rows":
        more = dict(total_tokens=s["k"].shape[0])
    if c["op"] == "attn":
        more = dict(total_tokens=s["q"].shape[0], max_new_tokens=max(s["new"]))
    if c["op"] == "evict":
        more = dict(budget=c["budget"], sink=c["sink"], recent=c["recent"], max_dst_pages=s["dst"].shape[1])
    make = lambda **kw: cosa.make_kv_params(num_reqs=c["reqs"], num_q_heads=c["q_heads"], num_kv_heads=c["kv_heads"],  # noqa: E731
                                            head_dim=c["d"], page_size=c["page"], num_pages=n16, num_kv4_pages=n4, **kw)
    s["p"] = make(max_seqlen=top, max_pages_per_req=pages, **more)
    if c["op"] == "attn":
        s["ws"] = torch.empty(cosa.cosa_kv4_attention_workspace_size(s["p"], with_weights=c["weights"]), dtype=torch.uint8, device=DEV)
    if c["op"] == "evict":
        s["p_back"] = make(max_seqlen=s["dst"].shape[1] * c["page"], max_pages_per_req=s["dst"].shape[1])


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "store": _own_store, "load": _own_load, "attn": _own_attn, "evict": _own_evict}[op](s)
    return {"rope": _rope, "store": _store, "load": _load, "attn": _attn, "evict": _evict}[op](s)


def _own_rope(s):
    from block_sparse_long_gb300 import kv as cosa

    if s["case"]["to"] == "pages":
        cosa.cosa_qk_norm_rope(s["p"], s["q"], s["k"], s["cu"], s["inv"], v=s["v"], q_weight=s["wq"], k_weight=s["wk"],
                               positions=s["pos"], start=s["start"], q_out=s["q_out"], k_cache=s["k_cache"],
                               v_cache=s["v_cache"], page_table=s["pt"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    cosa.cosa_qk_norm_rope(s["p"], s["q"], s["k"], s["cu"], s["inv"], q_weight=s["wq"], k_weight=s["wk"],
                           positions=s["pos"], q_out=s["q_out"], k_out=s["k_out"])
    return [s["q_out"], s["k_out"]]


def _own_store(s):
    from block_sparse_long_gb300 import kv as cosa

    if s["case"]["form"] == "rows":
        cosa.cosa_kv4_store(s["p"], s["cache"], s["pt"], s["k"], s["v"], cu_seqlens=s["cu"], start=s["start"])
    else:
        cosa.cosa_kv4_store(s["p"], s["cache"], s["pt"], s["k16"], s["v16"], src_page_table=s["pt16"], start=s["start"],
                            kv_len=s["kv_len"])
    return _own_load(s)


def _own_load(s):
    from block_sparse_long_gb300 import kv as cosa

    cosa.cosa_kv4_load(s["p"], s["cache"], s["pt"], s["k_back"], s["v_back"], s["pt16"], kv_len=s["kv_len"], start=s["start"])
    return [s["k_back"], s["v_back"]]


def _own_attn(s):
    from block_sparse_long_gb300 import kv as cosa

    cosa.cosa_kv4_attention(s["p"], s["q"], s["cu_q"], s["cache"], s["pt"], s["kv_len"], out=s["out"], weights=s["acc"],
                            workspace=s["ws"])
    return [s["out"]] if s["acc"] is None else [s["out"], s["acc"]]


def _own_evict(s):
    from block_sparse_long_gb300 import kv as cosa

    cosa.cosa_kv4_evict(s["p"], s["cache"], s["pt"], s["kv_len"], s["acc"], s["dst"], new_len=s["new_len"], kept=s["kept"],
                        weights_out=s["acc_out"])
    cosa.cosa_kv4_load(s["p_back"], s["cache"], s["dst"], s["k_back"], s["v_back"], s["pt16"], kv_len=s["new_len"])
    return [s["new_len"], s["kept"], s["acc_out"], s["k_back"], s["v_back"]]


# ---- plain forms ----
def _norm_rotate(x, w, pos, inv, interleaved):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    angle = (pos.double()[:, None] * inv)[:, None, :]            # far positions: the angle in 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    rot = 2 * inv.numel()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1).to(torch.bfloat16)


def _places(cu, start, table, P, T):
    """Flat page slots [T] of rows packed by cu, the first of each request at its start."""
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    at = (t - cu[b] + start[b]).long()
    return table[b, at // P].long() * P + at % P


def _rope(s):
    c = s["case"]
    s["q_out"].copy_(_norm_rotate(s["q"], s["wq"], s["pos"], s["inv"], c["interleaved"]))
    k = _norm_rotate(s["k"], s["wk"], s["pos"], s["inv"], c["interleaved"])
    if c["to"] != "pages":
        s["k_out"].copy_(k)
        return [s["q_out"], s["k_out"]]
    at = _places(s["cu"], s["start"], s["pt"], c["page"], k.shape[0])
    s["k_cache"].flatten(0, 1)[at] = k
    s["v_cache"].flatten(0, 1)[at] = s["v"]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _covered(s, table):
    """Flat page slots of every covered slot of the batch, request after request."""
    P = s["case"]["page"]
    a, e = s["start"].long(), s["kv_len"].long()
    n = e - a
    first = n.cumsum(0) - n
    b = torch.repeat_interleave(torch.arange(len(s["lens"]), device=DEV), n)
    at = torch.arange(b.numel(), device=DEV) - first[b] + a[b]
    return table[b, at // P].long() * P + at % P


def _store(s):
    to = _covered(s, s["pt16"])
    if s["case"]["form"] == "rows":
        k, v = s["k"], s["v"]
    else:
        k, v = s["k16"].flatten(0, 1)[to], s["v16"].flatten(0, 1)[to]
    for x, back in ((k, s["k_back"]), (v, s["v_back"])):
        u, sc = _quantise(x.float())
        y = u.unflatten(-1, (-1, GROUP)) * sc.float().unsqueeze(-1)
        back.flatten(0, 1)[to] = y.flatten(-2).to(torch.bfloat16)
    return [s["k_back"], s["v_back"]]


def _load(s):
    k, v = _unpack(s["cache"][s["pt"].long().flatten()], s["case"]["d"])
    P, pages = s["case"]["page"], s["pt"].shape[1]
    a, e = s["start"].long(), s["kv_len"].long()
    at = torch.arange(pages * P, device=DEV)
    fits = ((at >= a[:, None]) & (at < e[:, None])).flatten()
    to = (s["pt16"].long().repeat_interleave(P, 1) * P + at % P).flatten()[fits]
    for x, back in ((k, s["k_back"]), (v, s["v_back"])):
        back.flatten(0, 1)[to] = x.flatten(0, 1)[fits].to(torch.bfloat16)
    return [s["k_back"], s["v_back"]]


def _attn(s):
    c = s["case"]
    B, Hq, Hkv, d, P = c["reqs"], c["q_heads"], c["kv_heads"], c["d"], c["page"]
    k, v = _unpack(s["cache"][s["pt"].long().flatten()], d)
    S = s["pt"].shape[1] * P
    k, v = k.reshape(B, S, Hkv, d).transpose(1, 2), v.reshape(B, S, Hkv, d).transpose(1, 2)
    n, most = s["cu_q"].diff().long(), max(s["new"])
    i = torch.arange(most, device=DEV)
    there = i < n[:, None]                                        # [B, most]
    row = (s["cu_q"][:-1].long()[:, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][row].float().reshape(B, most, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    logit = q @ k.transpose(-1, -2) / math.sqrt(d)                # [B, Hkv, most * g, S]
    end = (s["kv_len"].long()[:, None] - n[:, None] + i + 1) * there
    seen = torch.arange(S, device=DEV) < end.repeat_interleave(Hq // Hkv, 1)[:, None, :, None]
    logit = logit.masked_fill(~seen, -math.inf)
    p = (logit - logit.amax(-1, keepdim=True).clamp_min(-1e30)).exp()
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = (p @ v).reshape(B, Hkv, most, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, most, Hq, d)
    s["out"][row[there]] = o[there].to(torch.bfloat16)
    if s["acc"] is None:
        return [s["out"]]
    s["acc"] += p.sum(2)
    return [s["out"], s["acc"]]


def _evict(s):
    c = s["case"]
    B, Hkv, P, d = c["reqs"], c["kv_heads"], c["page"], c["d"]
    S = s["pt"].shape[1] * P
    n = s["kv_len"].long()[:, None, None]
    at = torch.arange(S, device=DEV)
    w = s["acc"].masked_fill((at < c["sink"]) | (at >= n - c["recent"]), math.inf).masked_fill(at >= n, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., : c["budget"]]
    order = torch.nn.functional.pad(order, (0, c["budget"] - order.shape[-1]), value=S)
    most = torch.arange(c["budget"], device=DEV)
    left = n.clamp_max(c["budget"])
    kept = order.masked_fill(most >= left, S).sort(-1).values     # [B, Hkv, budget], S where there is none
    s["new_len"].copy_(left.flatten())
    s["kept"].copy_(kept.masked_fill(kept == S, -1))
    got = kept.clamp_max(S - 1)
    s["acc_out"].zero_()
    s["acc_out"][..., : c["budget"]] = s["acc"].gather(-1, got).masked_fill(kept == S, 0)[..., :S]
    k, v = _unpack(s["cache"][s["pt"].long().flatten()], d)
    fits = (most < left.flatten()[:, None]).flatten()
    to = (s["pt16"][:, most // P].long() * P + most % P).flatten()[fits]
    for x, back in ((k, s["k_back"]), (v, s["v_back"])):
        x = x.reshape(B, S, Hkv, d).transpose(1, 2).gather(2, got[..., None].expand(-1, -1, -1, d)).transpose(1, 2)
        back.flatten(0, 1)[to] = x.flatten(0, 1)[fits].to(torch.bfloat16)
    return [s["new_len"], s["kept"], s["acc_out"], s["k_back"], s["v_back"]]


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, request by request
# ---------------------------------------------------------------------------------------------------------------
def _code_index(d):
    """Byte offset and nibble of value j of a K row and of a V row, from the layout's words."""
    G = d // GROUP
    j = torch.arange(d)
    g, r = j // GROUP, j % GROUP
    k_nib = ((r // 8) * G + g) * 8 + r % 8
    v_nib = ((r // 4) * G + g) * 4 + r % 4
    return k_nib.to(DEV), v_nib.to(DEV)


def _exact_values(cache, pages, n, d):
    """Slots 0..n-1 of one request: float64 K, V [n, H, d]."""
    P = cache.shape[2]
    tile = cache[pages.long()].reshape(len(pages), cache.shape[1], P // 16, 18 * d).transpose(1, 2).flatten(0, 1)
    slot = torch.arange(n, device=DEV)
    rows, t = tile[slot // 16], slot % 16                          # [n, H, 18 d]
    kn, vn = _code_index(d)
    G = d // GROUP
    got = []
    for nib, base, row, sbase in ((kn, 0, t, 16 * d), (vn, 8 * d, (t % 2) * 8 + t // 2, 16 * d + 32 * G)):
        def nibble(n):
            byte = base + row[:, None] * (d // 2) + n // 2
            b = rows.gather(2, byte[:, None, :].expand(-1, rows.shape[1], -1))
            return torch.where((n % 2).bool(), b >> 4, b & 15).double()

        sign = 1 - 2 * torch.floor(nibble(nib ^ 2) / 8)
        code = torch.remainder(nibble(nib), 8) * sign
        at = sbase + t[:, None] * 2 * G + torch.arange(G, device=DEV) * 2
        lo = rows.gather(2, at[:, None, :].expand(-1, rows.shape[1], -1)).int()
        hi = rows.gather(2, at[:, None, :].expand(-1, rows.shape[1], -1) + 1).int()
        scale = ((hi << 24) | (lo << 16)).view(torch.float32).double()
        got.append(code * scale.repeat_interleave(GROUP, -1))
    return got


def _put(back, pages, first, x):
    P = back.shape[1]
    at = torch.arange(first, first + x.shape[0], device=DEV)
    back.flatten(0, 1)[pages.long()[at // P] * P + at % P] = x


def exact(c, seed):
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    op, lens, d, P = c["op"], s["lens"], c["d"], c["page"]
    if op == "rope":
        return _exact_rope(c, s)
    if op in ("store", "load"):
        kb, vb = s["k_back"].double(), s["v_back"].double()
        row = 0
        for b, (a, e) in enumerate(s["slots"]):
            if op == "load":
                k, v = (x[a:] for x in _exact_values(s["cache"], s["pt"][b], e, d))
            else:
                if c["form"] == "rows":
                    k, v = s["k"][row:row + e - a], s["v"][row:row + e - a]
                    row += e - a
                else:
                    at = torch.arange(a, e, device=DEV)
                    at = s["pt16"][b].long()[at // P] * P + at % P
                    k, v = s["k16"].flatten(0, 1)[at], s["v16"].flatten(0, 1)[at]
                k, v = _exact_round(k.double()), _exact_round(v.double())
            _put(kb, s["pt16"][b], a, k)
            _put(vb, s["pt16"][b], a, v)
        return [kb, vb]
    if op == "attn":
        return _exact_attn(c, s)
    # evict: a slot's place in the order is how many slots beat it
    kb, vb = s["k_back"].double(), s["v_back"].double()
    acc = torch.zeros_like(s["acc"], dtype=torch.float64)
    for b, n in enumerate(lens):
        k, v = _exact_values(s["cache"], s["pt"][b], n, d)
        left = min(n, c["budget"])
        must = torch.zeros(n, dtype=torch.bool, device=DEV)
        must[: c["sink"]] = True
        must[max(0, n - c["recent"]):] = True
        for h in range(c["kv_heads"]):
            w = s["acc"][b, h, :n].double()
            key = torch.where(must, torch.full_like(w, 1e300), w)
            bar = key.sort(descending=True).values[left - 1]
            sure = key > bar
            ties = (key == bar).nonzero().flatten()[: left - int(sure.sum())]
            sure[ties] = True
            kept = sure.nonzero().flatten()
            acc[b, h, :left] = w[kept]
            at = torch.arange(left, device=DEV)
            at = s["pt16"][b].long()[at // P] * P + at % P
            kb.flatten(0, 1)[at, h] = k[kept, h]
            vb.flatten(0, 1)[at, h] = v[kept, h]
    return [None, None, acc, kb, vb]


def _exact_round(x):
    """The values a 4-bit store keeps: the scale is the bf16 nearest to max/7, the code the nearest whole multiple."""
    g = x.unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).double()
    code = torch.round(g / torch.where(scale == 0, torch.ones_like(scale), scale)).clamp(-7, 7)
    return (code * scale).flatten(-2)


def _exact_rope(c, s):
    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        y = x.clone()
        for i in range(c["rot"] // 2):
            lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rot"] // 2)
            a = (s["pos"].double() * s["inv"][i])[:, None]
            y[..., lo] = x[..., lo] * torch.cos(a) - x[..., hi] * torch.sin(a)
            y[..., hi] = x[..., lo] * torch.sin(a) + x[..., hi] * torch.cos(a)
        return y

    d, P = c["d"], c["page"]
    q, k = turned(s["q"], s["wq"]), turned(s["k"], s["wk"])
    if c["to"] != "pages":
        return [q, k]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    row = 0
    for b, n in enumerate(s["lens"]):
        _put(kc, s["pt"][b], int(s["start"][b]), k[row:row + n])
        _put(vc, s["pt"][b], int(s["start"][b]), s["v"][row:row + n].double())
        row += n
    return [q, kc, vc]


def _exact_attn(c, s):
    d, g = c["d"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    acc = None if s["acc"] is None else s["acc"].double()
    row = 0
    for b, n in enumerate(s["lens"]):
        k, v = _exact_values(s["cache"], s["pt"][b], n, d)
        for j in range(s["new"][b]):
            end = n - s["new"][b] + j + 1
            q = s["q"][row + j].double().reshape(c["kv_heads"], g, d)
            p = torch.softmax(torch.einsum("hgd,shd->hgs", q, k[:end]) / math.sqrt(d), -1)
            out[row + j] = torch.einsum("hgs,shd->hgd", p, v[:end]).reshape(-1, d)
            if acc is not None:
                acc[b, :, :end] += p.sum(1)
        row += s["new"][b]
    return [out] if acc is None else [out, acc]
