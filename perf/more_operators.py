"""Attention of drafted tokens and over latent vectors, each operator in its plain form and as the library's call.

  tree     attention of a tree of drafted tokens per request over the bf16 pages of the sparse prefill (single new tokens and
           chains of them are trees too)
  commit   the accepted path of each tree moved, in place, to the slots behind its context
  rope     latent vector of every token normed, its shared key part and the queries' parts rotated, the key written to
           pages of latent vectors (and to rows, from which a prompt's keys and values are expanded)
  latent   attention of new tokens over the pages of latent vectors: a token's vector of latent_dim + 64 values is the key of
           every head, its first latent_dim values are the value (the absorbed form)
  expand   causal attention of prompts in the expanded form: per head a key of d values and a value of d values, and 64
           rotated key values that all heads share

`own` chooses between the plain form (torch operations in 32 bits) and the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"
ROT = 64  # rotated values of a latent key


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _lens(c):
    """Request lengths of a case: the first is the longest, the others spread between the bounds."""
    r = random.Random(c["len_seed"])
    return [c["max_len"]] + [r.randint(c["min_len"], c["max_len"]) for _ in range(c["reqs"] - 1)]


def _nodes(c):
    """New tokens of each request: the first has the most."""
    r = random.Random(c["len_seed"] + 1)
    return [c["nodes"]] + [r.randint(1, c["nodes"]) for _ in range(c["reqs"] - 1)]


def listed():
    gqa = dict(q_heads=32, kv_heads=8, d=128, page=64)
    return [
        # one new token of one short conversation over the prompt's bf16 pages: latency
        dict(name="tree 1x900 token", op="tree", reqs=1, min_len=900, max_len=900, nodes=1, tree=False, lse=False, len_seed=1, **gqa),
        # a serving batch in which every request checks a drafted tree of up to 13 tokens
        dict(name="tree 24 ragged 13", op="tree", reqs=24, min_len=1000, max_len=16384, nodes=13, tree=True, lse=True, len_seed=2, **gqa),
        # the benchmark's 128K context with the widest tree, 64 tokens: 256 query rows a kv head
        dict(name="tree 1x128k 64", op="tree", reqs=1, min_len=131072, max_len=131072, nodes=64, tree=True, lse=False, len_seed=3, **gqa),
        # after the check: what 64 requests accepted of their trees, in keys and values
        dict(name="commit 64", op="commit", cache="pages", reqs=64, min_len=100, max_len=1000, nodes=40, len_seed=4, **gqa),
        # the same of one request's latent vectors
        dict(name="commit 1 latent", op="commit", cache="latent", reqs=1, min_len=500, max_len=500, nodes=20, len_seed=5, page=16, latent=512),
        # a decode step of 64 requests: one new token each into its page
        dict(name="rope decode 64", op="rope", reqs=64, min_len=1, max_len=1, ctx=6000, heads=32, latent=512, page=64, interleaved=True,
             rows=False, norm=True, len_seed=6),
        # the prompts of a batch, 40K tokens at most, into pages and into rows for the expansion
        dict(name="rope 3 prompts", op="rope", reqs=3, min_len=5000, max_len=13333, ctx=0, heads=32, latent=512, page=64, interleaved=False,
             rows=True, norm=True, len_seed=7),
        # one new token of one short conversation, sixteen heads over one latent vector: latency
        dict(name="latent 1x900 token", op="latent", reqs=1, min_len=900, max_len=900, nodes=1, tree=False, lse=False, heads=16, latent=512,
             page=64, len_seed=8),
        # one 128K context, one new token: the cache is read by the whole card
        dict(name="latent 1x128k token", op="latent", reqs=1, min_len=131072, max_len=131072, nodes=1, tree=False, lse=False, heads=32,
             latent=512, page=64, len_seed=9),
        # a serving batch with drafted trees of up to seven tokens: up to 224 query rows over each vector
        dict(name="latent 24 ragged 7", op="latent", reqs=24, min_len=1000, max_len=16384, nodes=7, tree=True, lse=True, heads=32, latent=512,
             page=64, len_seed=10),
        # a ragged batch of prompts, heads of 64, each behind 333 tokens that are there already
        dict(name="expand 5 ragged d64", op="expand", reqs=5, min_len=37, max_len=2011, ctx=333, heads=6, d=64, lse=True, len_seed=11),
        # a 16K-token prompt's attention, heads of 128 + 64
        dict(name="expand 16k", op="expand", reqs=1, min_len=16384, max_len=16384, ctx=0, heads=16, d=128, lse=False, len_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "commit", "rope", "latent", "latent", "expand"))
    c = dict(op=op, len_seed=rng.randrange(1 << 30), page=rng.choice((16, 32, 64, 128)))
    kv = rng.choice((1, 2, 4, 8))
    gqa = dict(q_heads=kv * rng.choice((1, 2, 3, 4, 7, 8) if kv < 8 else (1, 2, 3, 4)), kv_heads=kv, d=rng.choice((64, 128)))
    reqs = _log(rng, 1, 64)
    if op == "expand":
        reqs = _log(rng, 1, 8)
        heads, d = rng.choice((1, 2, 3, 5, 8, 16)), rng.choice((64, 128))
        # pairs of the whole batch at most: below the largest listed case
        top = _log(rng, 1, math.sqrt((1 << 28) / reqs * 16 / heads / 4))
        c.update(heads=heads, d=d, ctx=rng.choice((0, 0, rng.randint(1, 1 + top // 2))), lse=rng.random() < 0.5)
    elif op == "rope":
        top = _log(rng, 1, (1 << 15) // reqs)
        c.update(heads=rng.choice((1, 5, 8, 16, 20, 32)), latent=rng.choice((256, 512)), ctx=rng.randint(0, 2000),
                 interleaved=rng.random() < 0.5, rows=rng.random() < 0.5, norm=rng.random() < 0.8)
    elif op == "commit":
        top = _log(rng, 1, 1000)
        c.update(cache=rng.choice(("pages", "latent")), nodes=rng.randint(1, min(64, top)), latent=rng.choice((256, 512)), **gqa)
    else:
        top = _log(rng, 1, (1 << 17) // reqs)
        nodes = min(top, rng.choice((1, 1, 1, 2, 3, 5, 8, rng.randint(1, 64))))
        if op == "latent":
            heads = rng.choice((1, 8, 16, 16, 32, 32, 20, 64, 128))
            nodes = max(1, min(nodes, 224 // heads))
            c.update(heads=heads, latent=rng.choice((256, 512, 512)))
        else:
            c.update(**gqa)
        c.update(nodes=nodes, tree=rng.random() < 0.6, lse=rng.random() < 0.5)
    c.update(reqs=reqs, max_len=top, min_len=rng.randint(min(top, c.get("nodes", 1)), top))
    return c


def _pairs(c):
    """Query-key pairs of the causal prompts (each prompt behind ctx tokens that are there already)."""
    return sum(n * c["ctx"] + n * (n + 1) // 2 for n in _lens(c))


def work(c):
    lens, op = _lens(c), c["op"]
    n = sum(lens)
    if op == "expand":
        rows = 2 * c["heads"] * (c["d"] + ROT) * n + 2 * (n + c["reqs"] * c["ctx"]) * (2 * c["heads"] * c["d"] + ROT)
        return {"bytes": rows + 2 * n * c["heads"] * c["d"], "flops": 2 * _pairs(c) * c["heads"] * (2 * c["d"] + ROT)}
    if op == "rope":
        kv = 2 * (c["latent"] + ROT)
        return {"bytes": n * (2 * kv + (kv if c["rows"] else 0) + 4 * c["heads"] * ROT),
                "flops": n * (4 * c["latent"] + 3 * ROT * (1 + c["heads"]))}
    if op == "commit":
        moved = sum(sum(i != j for i, j in enumerate(p)) for p in _trees(c)[1])
        return {"bytes": max(64, 2 * moved * 2 * _row(c) * (2 if c["cache"] == "pages" else 1)), "flops": 0}
    new = _nodes(c)
    if op == "latent":
        wide = c["latent"] + ROT
        return {"bytes": 2 * n * wide + 2 * sum(new) * c["heads"] * (wide + c["latent"]),
                "flops": 2 * sum(m * v for m, v in zip(new, lens)) * c["heads"] * (wide + c["latent"])}
    return {"bytes": 4 * n * c["kv_heads"] * c["d"] + 4 * sum(new) * c["q_heads"] * c["d"],
            "flops": 4 * sum(m * v for m, v in zip(new, lens)) * c["q_heads"] * c["d"]}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    return _i32([0] + [sum(lens[: i + 1]) for i in range(len(lens))])


def _table(g, reqs, pages):
    """A shuffled page table [reqs, pages]."""
    return torch.randperm(reqs * pages, generator=g, device=DEV).to(torch.int32).reshape(reqs, pages)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _row(c):
    """Values of a cache's row."""
    return c["latent"] + ROT if c["op"] == "commit" and c["cache"] == "latent" else c["kv_heads"] * c["d"]


def _trees(c):
    """Random trees, node by node behind its parent: per request the masks (bit j: node j is the node or above it) and one
    path from the top, as an accepted draft has."""
    r = random.Random(c["len_seed"] + 2)
    masks, paths = [], []
    for n in _nodes(c):
        up = [r.randint(-1, i - 1) if r.random() < 0.5 else i - 1 for i in range(n)]
        m = []
        for i, p in enumerate(up):
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        end = r.randrange(n)
        masks.append(m)
        paths.append([j for j in range(n) if m[end] >> j & 1])
    return masks, paths


def _bits(masks):
    flat = [m - (1 << 64) if m >> 63 else m for req in masks for m in req]
    return torch.tensor(flat, dtype=torch.int64, device=DEV)


def prepare(c, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    op, B, lens = c["op"], c["reqs"], _lens(c)
    s = dict(case=c, lens=lens)
    if op == "expand":
        H, d, T = c["heads"], c["d"], sum(lens)
        s["total"] = [n + c["ctx"] for n in lens]
        s["cu"], s["cu_kv"] = _cu(lens), _cu(s["total"])
        q = _normal(g, T, H * (d + ROT)).unflatten(1, (H, d + ROT))     # a row of the query projection
        kv = _normal(g, sum(s["total"]), H * 2 * d).unflatten(1, (H, 2 * d))      # and of the expansion: keys, values
        s["q"], s["q_rope"] = q[..., :d], q[..., d:].contiguous()
        s["k"], s["v"] = kv[..., :d], kv[..., d:]
        s["k_rope"] = _normal(g, sum(s["total"]), ROT)
        s["out"] = torch.zeros(T, H, d, dtype=torch.bfloat16, device=DEV)
        s["scale"] = (d + ROT) ** -0.5
        if c["lse"]:
            s["lse"] = torch.zeros(T, H, device=DEV)
    elif op == "rope":
        H, T, P, DL = c["heads"], sum(lens), c["page"], c["latent"]
        s["cu"] = _cu(lens)
        s["kv"] = _normal(g, T, DL + ROT)
        s["q"] = _normal(g, T, H * (128 + ROT)).unflatten(1, (H, 128 + ROT))[..., 128:]
        s["w"] = (1 + 0.2 * _normal(g, DL)) if c["norm"] else None
        s["inv"] = 1e6 ** (-torch.arange(0, ROT, 2, device=DEV, dtype=torch.float64) / ROT)
        start = [c["ctx"] + (7 * b) % 101 for b in range(B)]
        s["start"] = _i32(start)
        pages = -(-max(f + n for f, n in zip(start, lens)) // P)
        s["pt"] = _table(g, B, pages)
        s["cache"] = torch.zeros(B * pages, P, DL + ROT, dtype=torch.bfloat16, device=DEV)
        s["q_out"] = torch.zeros(T, H, ROT, dtype=torch.bfloat16, device=DEV)
        if c["rows"]:
            s["c_out"] = torch.zeros(T, DL, dtype=torch.bfloat16, device=DEV)
            s["k_out"] = torch.zeros(T, ROT, dtype=torch.bfloat16, device=DEV)
    else:
        P, pages = c["page"], -(-c["max_len"] // c["page"])
        masks, paths = _trees(c)
        new = [min(m, n) for m, n in zip(_nodes(c), lens)]
        masks, paths = [m[:k] for m, k in zip(masks, new)], [[j for j in p if j < k] for p, k in zip(paths, new)]
        s["cu"], s["kv_len"], s["new"], s["pt"] = _cu(new), _i32(lens), new, _table(g, B, pages)
        T = sum(new)
        if op == "commit":
            wide = [(_row(c),)] if c["cache"] == "latent" else [(c["kv_heads"], c["d"])] * 2
            s["caches"] = [_normal(g, B * pages, P, *w) for w in wide]
            s["path"] = _i32([p + [-1] * (c["nodes"] - len(p)) for p in paths])
            s["path_len"], s["new_len"] = _i32([len(p) for p in paths]), torch.zeros(B, dtype=torch.int32, device=DEV)
        elif op == "latent":
            H, DL = c["heads"], c["latent"]
            s["cache"] = _normal(g, B * pages, P, DL + ROT)
            s["q"], s["q_rope"] = _normal(g, T, H, DL), _normal(g, T, H, ROT)
            s["out"], s["scale"] = torch.zeros_like(s["q"]), (128 + ROT) ** -0.5
        else:
            s["k"], s["v"] = (_normal(g, B * pages, P, c["kv_heads"], c["d"]) for _ in range(2))
            s["q"] = 1.5 * _normal(g, T, c["q_heads"], c["d"])
            s["out"], s["scale"] = torch.zeros_like(s["q"]), c["d"] ** -0.5
        if op != "commit":
            s["mask"] = _bits(masks) if c["tree"] else None
            if c["lse"]:
                s["lse"] = torch.zeros(s["q"].shape[:2], device=DEV)
    if own:
        _plan(s)
    return s


def _plan(s):
    """The library's parameters and workspace, which a program makes once for its shapes."""
    from block_sparse_long_gb300 import attn as cosa

    c = s["case"]
    op = c["op"]
    more = dict(num_reqs=c["reqs"], total_tokens=sum(s.get("new", s["lens"])))
    if op == "expand":
        more.update(num_q_heads=c["heads"], head_dim=c["d"], total_kv_tokens=sum(s["total"]), max_new_tokens=max(s["lens"]), sm_scale=s["scale"])
    else:
        pages = s["pt"].shape[1]
        more.update(page_size=c["page"], max_pages_per_req=pages, max_seqlen=pages * c["page"], num_pages=c["reqs"] * pages)
    if op == "rope":
        more.update(num_q_heads=c["heads"], latent_dim=c["latent"], interleaved=c["interleaved"])
    elif op == "commit":
        more.update(num_q_heads=1, max_new_tokens=c["nodes"])
    elif op in ("tree", "latent"):
        more.update(max_new_tokens=max(s["new"]), sm_scale=s["scale"])
        more.update(dict(num_q_heads=c["heads"], latent_dim=c["latent"]) if op == "latent" else
                    dict(num_q_heads=c["q_heads"], num_kv_heads=c["kv_heads"], head_dim=c["d"]))
    s["p"] = cosa.make_attn_params(**more)
    if op == "tree":
        s["ws"] = torch.empty(max(1, cosa.cosa_tree_attention_workspace_size(s["p"])), dtype=torch.uint8, device=DEV)
    if op == "latent":
        s["ws"] = torch.empty(max(1, cosa.cosa_latent_attention_workspace_size(s["p"])), dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        _own(s)
    else:
        {"tree": _tree, "commit": _commit, "rope": _rope, "latent": _latent, "expand": _expand}[op](s)
    if op == "commit":
        return [*s["caches"], s["new_len"]]
    if op == "rope":
        return [s["q_out"], s["cache"]] + ([s["c_out"], s["k_out"]] if "c_out" in s else [])
    return [s["out"]] + ([s["lse"]] if "lse" in s else [])


def _own(s):
    from block_sparse_long_gb300 import attn as cosa

    op = s["case"]["op"]
    if op == "tree":
        cosa.cosa_tree_attention(s["p"], s["q"], s["cu"], s["k"], s["v"], s["pt"], s["kv_len"], tree_mask=s["mask"], out=s["out"],
                                 lse=s.get("lse"), workspace=s["ws"])
    elif op == "commit":
        cosa.cosa_tree_commit(s["p"], s["caches"], s["cu"], s["pt"], s["kv_len"], s["path"], s["path_len"], new_len=s["new_len"])
    elif op == "rope":
        cosa.cosa_latent_rope(s["p"], s["kv"], s["cu"], s["inv"], q=s["q"], weight=s["w"], start=s["start"], q_out=s["q_out"],
                              c_out=s.get("c_out"), k_out=s.get("k_out"), cache=s["cache"], page_table=s["pt"])
    elif op == "latent":
        cosa.cosa_latent_attention(s["p"], s["q"], s["q_rope"], s["cu"], s["cache"], s["pt"], s["kv_len"], tree_mask=s["mask"],
                                   out=s["out"], lse=s.get("lse"), workspace=s["ws"])
    else:
        cosa.cosa_latent_prefill(s["p"], s["q"], s["q_rope"], s["k"], s["k_rope"], s["v"], s["cu"], cu_kv=s["cu_kv"], out=s["out"],
                                 lse=s.get("lse"))


# ---- plain forms ----
def _request(s, cache, b):
    """Slots of request b: [pages * P, ...] in 32 bits."""
    n = s["lens"][b]
    return cache[s["pt"][b].long()].flatten(0, 1)[:n].float()


def _seen(s, b):
    """[new, kv_len]: what each new token of request b attends to."""
    n, m = s["lens"][b], s["new"][b]
    at, i = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
    if s["mask"] is None:
        return at <= n - m + i[:, None]
    bits = s["mask"][sum(s["new"][:b]):][:m]
    tail = (bits[:, None] >> i) & 1
    return torch.cat((torch.ones(m, n - m, dtype=torch.bool, device=DEV), tail.bool()), 1)


def _softmax(logit, seen):
    """Weights and log of the sum; a row that sees nothing has no weight."""
    logit = logit.masked_fill(~seen, -math.inf)
    top = logit.amax(-1, keepdim=True).clamp_min(-1e30)
    p = (logit - top).exp()
    total = p.sum(-1, keepdim=True)
    return p / total.clamp_min(1e-30), (top + total.log()).squeeze(-1)


def _put(s, b, o, lse):
    row = sum(s["new"][:b])
    s["out"][row:row + o.shape[0]] = o.to(torch.bfloat16)
    if "lse" in s:
        s["lse"][row:row + o.shape[0]] = lse


def _tree(s):
    c = s["case"]
    Hkv, group = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    for b, m in enumerate(s["new"]):
        k, v = (_request(s, x, b).transpose(0, 1) for x in (s["k"], s["v"]))          # [Hkv, n, d]
        q = s["q"][sum(s["new"][:b]):][:m].float().unflatten(1, (Hkv, group)).permute(1, 0, 2, 3).flatten(1, 2)
        p, lse = _softmax(q @ k.transpose(1, 2) * s["scale"], _seen(s, b).repeat_interleave(group, 0))
        o = (p @ v).unflatten(1, (m, group)).transpose(0, 1).flatten(1, 2)
        _put(s, b, o, lse.unflatten(1, (m, group)).transpose(0, 1).flatten(1, 2))


def _latent(s):
    c = s["case"]
    for b, m in enumerate(s["new"]):
        k = _request(s, s["cache"], b)
        row = sum(s["new"][:b])
        q = torch.cat((s["q"][row:row + m], s["q_rope"][row:row + m]), -1).float()     # [m, H, latent + 64]
        p, lse = _softmax((q.flatten(0, 1) @ k.T).unflatten(0, q.shape[:2]) * s["scale"], _seen(s, b)[:, None, :])
        _put(s, b, (p.flatten(0, 1) @ k[:, :c["latent"]]).unflatten(0, q.shape[:2]), lse)


def _expand(s):
    c = s["case"]
    H = c["heads"]
    row = at = 0
    for n, total in zip(s["lens"], s["total"]):
        seen = torch.arange(total, device=DEV) <= total - n + torch.arange(n, device=DEV)[:, None]
        heads = max(1, (1 << 28) // (n * total))           # heads whose logits are held at once
        for h in range(0, H, heads):
            few = slice(h, h + heads)
            q = torch.cat((s["q"][row:row + n, few], s["q_rope"][row:row + n, few]), -1).float().transpose(0, 1)
            k = s["k"][at:at + total, few].float()
            k = torch.cat((k, s["k_rope"][at:at + total, None].float().expand(-1, k.shape[1], -1)), -1).permute(1, 2, 0)
            p, lse = _softmax(q @ k * s["scale"], seen)
            s["out"][row:row + n, few] = (p @ s["v"][at:at + total, few].float().transpose(0, 1)).transpose(0, 1).to(torch.bfloat16)
            if "lse" in s:
                s["lse"][row:row + n, few] = lse.T
        row, at = row + n, at + total


def _rotate(x, pos, inv, interleaved):
    angle = (pos.double()[:, None] * inv)            # far positions: the angle in 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    while cos.dim() < x.dim():
        cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _rope(s):
    c = s["case"]
    T, DL, P = s["kv"].shape[0], c["latent"], c["page"]
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    slot = (t - s["cu"][b] + s["start"][b]).long()
    x = s["kv"][:, :DL].float()
    if s["w"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    x = x.to(torch.bfloat16)
    k = _rotate(s["kv"][:, DL:].float(), slot, s["inv"], c["interleaved"]).to(torch.bfloat16)
    s["q_out"].copy_(_rotate(s["q"].float(), slot, s["inv"], c["interleaved"]))
    s["cache"].flatten(0, 1)[s["pt"][b, slot // P].long() * P + slot % P] = torch.cat((x, k), -1)
    if c["rows"]:
        s["c_out"].copy_(x)
        s["k_out"].copy_(k)


def _commit(s):
    c = s["case"]
    P, n, path = c["page"], s["path_len"].long(), s["path"].long()
    base = s["kv_len"].long() - s["cu"].diff().long()
    i = torch.arange(path.shape[1], device=DEV)
    taken = i < n[:, None]
    b = torch.arange(c["reqs"], device=DEV)[:, None].expand_as(path)[taken]
    src, dst = (base[:, None] + path)[taken], (base[:, None] + i)[taken]
    place = lambda at: s["pt"][b, at // P].long() * P + at % P  # noqa: E731
    for x in s["caches"]:
        flat = x.flatten(0, 1)
        flat[place(dst)] = flat[place(src)]
    s["new_len"].copy_(base + n)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, request by request
# ---------------------------------------------------------------------------------------------------------------
def exact(c, seed):
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    op, lens = c["op"], s["lens"]
    if op == "commit":
        return _exact_commit(c, s)
    if op == "rope":
        return _exact_rope(c, s)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=DEV)
    masks = _trees(c)[0] if op != "expand" else None
    row = at = 0
    for b, n in enumerate(lens):
        if op == "expand":
            new, total = n, s["total"][b]
            see = torch.ones(new, total, dtype=torch.bool, device=DEV).tril(total - new)
        else:
            new, total = s["new"][b], n
            see = torch.ones(new, total, dtype=torch.bool, device=DEV)
            for i in range(new):
                for j in range(new):
                    if not (masks[b][i] >> j & 1 if c["tree"] else j <= i):
                        see[i, total - new + j] = False
            slot = torch.arange(total, device=DEV)
            place = s["pt"][b].long()[slot // c["page"]], slot % c["page"]
        for h in range(out.shape[1]):
            if op == "expand":
                q = torch.cat((s["q"][row:row + new, h], s["q_rope"][row:row + new, h]), 1).double()
                k = torch.cat((s["k"][at:at + total, h], s["k_rope"][at:at + total]), 1).double()
                v = s["v"][at:at + total, h].double()
            elif op == "tree":
                q = s["q"][row:row + new, h].double()
                k, v = (x[place[0], place[1], h * c["kv_heads"] // c["q_heads"]].double() for x in (s["k"], s["v"]))
            else:
                q = torch.cat((s["q"][row:row + new, h], s["q_rope"][row:row + new, h]), 1).double()
                if h == 0:
                    k = s["cache"][place].double()
                    v = k[:, :c["latent"]]
            x = torch.einsum("id,jd->ij", q, k) * s["scale"]
            x[~see] = -math.inf
            lse[row:row + new, h] = torch.logsumexp(x, 1)
            out[row:row + new, h] = torch.softmax(x, 1) @ v
        row, at = row + new, at + total
    return [out, lse] if "lse" in s else [out]


def _exact_commit(c, s):
    caches = [x.double() for x in s["caches"]]
    paths = _trees(c)[1]
    for b, n in enumerate(s["lens"]):
        path = [j for j in paths[b] if j < s["new"][b]]
        base, page, pt = n - s["new"][b], c["page"], s["pt"][b].tolist()
        for x in caches:
            rows = [x[pt[(base + j) // page], (base + j) % page].clone() for j in path]
            for i, r in enumerate(rows):
                x[pt[(base + i) // page], (base + i) % page] = r
    return [*caches, None]


def _exact_rope(c, s):
    DL, P = c["latent"], c["page"]
    pos = torch.cat([torch.arange(int(f), int(f) + n, device=DEV) for f, n in zip(s["start"].tolist(), s["lens"])]).double()

    def turned(x):
        y = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        x = x.double()
        for i in range(ROT // 2):
            lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + ROT // 2)
            a = (pos * s["inv"][i]).reshape(-1, *[1] * (x.dim() - 2))
            y[..., lo] = x[..., lo] * torch.cos(a) - x[..., hi] * torch.sin(a)
            y[..., hi] = x[..., lo] * torch.sin(a) + x[..., hi] * torch.cos(a)
        return y

    x = s["kv"][:, :DL].double()
    if s["w"] is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / DL + 1e-6) * s["w"].double()
    k, cache = turned(s["kv"][:, DL:]), s["cache"].double()
    row = 0
    for b, n in enumerate(s["lens"]):
        slot = torch.arange(n, device=DEV) + int(s["start"][b])
        cache[s["pt"][b].long()[slot // P], slot % P] = torch.cat((x[row:row + n], k[row:row + n]), 1)
        row += n
    return [turned(s["q"]), cache] + ([x, k] if c["rows"] else [])
