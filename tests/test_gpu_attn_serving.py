"""libcosa_attn's calls as a serving loop uses them: together, on streams, in graphs, two at once, on large caches, on every path of
the launch rule, and with waits that run out."""
import time

import numpy as np
import pytest
import torch

from block_sparse_long_gb300 import attn as C, kv as K
from tests import attn_reference as ref
from tests.attn_helpers import DEV, Paged, bits, near
from tests.attn_paths import path, together
from tests.kv_helpers import bf, cu_of, i32, new_status, ok, table
from tests.kv_reference import bf16, norm_rope, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_long_gb300 import build
    build.build()


# ---------------------------------------------------------------------------------------------------------------
# every path
# ---------------------------------------------------------------------------------------------------------------
# path, lens, new, q heads, kv heads, latent, head_dim, tables for (slots or None)
PATHS = [
    ("whole", [100, 60, 128] * 30, [1] * 90, 8, 4, 0, 128, None),
    ("whole", [100, 60, 300] * 60, [1] * 180, 4, 1, 256, 128, None),
    ("cluster 2", [250, 200, 70], [1, 1, 1], 8, 4, 0, 64, None),
    ("cluster 4", [500, 400, 450], [2, 1, 2], 8, 2, 0, 128, None),
    ("cluster 8", [900, 1000], [5, 64], 8, 2, 0, 128, None),
    ("cluster 8", [1000], [64], 2, 1, 0, 64, None),
    ("cluster 4", [500, 400], [1, 3], 16, 1, 512, 128, None),
    ("cluster 8", [900, 8], [2, 4], 16, 1, 512, 128, None),
    ("cluster 8", [1000, 3], [3, 3], 8, 1, 256, 128, None),
    ("list, by item, wide", [20000, 100], [3, 1], 8, 2, 0, 128, None),
    ("list, by item, wide", [20000], [3], 8, 1, 512, 128, None),
    ("list, by item, wide", [20], [3], 8, 1, 512, 128, 40000),
    ("list, by item", [5000, 100, 3000, 2000, 900], [13, 2, 5, 3, 1], 32, 8, 0, 128, None),
    ("list, by item", [3000, 900, 5000, 70] * 11, [1, 2, 2, 1] * 11, 16, 1, 256, 128, None),
    ("list, by cta", [3000, 900, 2000, 70] * 4, [1, 3, 2, 7] * 4, 16, 8, 0, 64, None),
    ("list, by cta", [900, 2500, 70] * 40, [1, 2, 1] * 40, 16, 1, 512, 128, None),
]


@pytest.mark.parametrize("name,lens,new,Hq,Hkv,latent,d,slots", PATHS)
def test_every_path(name, lens, new, Hq, Hkv, latent, d, slots):
    c = Paged(len(lens) + Hq, lens, new, Hq, Hkv, d, 64, latent=latent, tree=True, pitch=None if slots is None else slots // 64)
    assert path(c.p, latent) == name
    for _ in range(2):
        out, lse = c.buffers()
        guard, st = out.clone(), new_status()
        c.call(out=out, lse=lse, status=st)
        ok(st)
        c.check(out, lse)
        assert torch.equal(out[c.T:], guard[c.T:])


# path, row tiles together, lens, new, hint, q heads, kv heads, tree
TOGETHER = [
    ("list, by item, wide", 2, [12000], [64], 64, 16, 4, True),
    ("list, by item", 2, [9000, 3000], [64, 63], 33, 16, 4, True),                 # twice as many as the hint says
    ("list, by item", 4, [9000, 3000, 700], [64, 64, 40], 64, 16, 2, True),        # the last has three row tiles
    ("list, by item", 7, [9000], [330], 330, 8, 1, False),                         # three rounds of seven for 21
    ("list, by cta", 3, [1900, 700] * 6, [38, 48] * 6, 48, 32, 4, True),
    ("whole", 2, [200] * 60, [40] * 60, 40, 16, 4, True),
]


@pytest.mark.parametrize("name,row_tiles,lens,new,hint,Hq,Hkv,tree", TOGETHER)
def test_row_tiles_together(name, row_tiles, lens, new, hint, Hq, Hkv, tree):
    c = Paged(len(lens) + Hq, lens, new, Hq, Hkv, 128, 64, tree=tree)
    c.p.max_new_tokens = hint
    assert (path(c.p, 0), together(c.p, 0)) == (name, row_tiles)
    for _ in range(2):
        out, lse = c.buffers()
        guard, st = out.clone(), new_status()
        c.call(out=out, lse=lse, status=st)
        ok(st)
        c.check(out, lse)
        assert torch.equal(out[c.T:], guard[c.T:])


@pytest.mark.parametrize("name,lens,new,Hq,Hkv,latent,d,slots", PATHS + [(name, lens, new, Hq, Hkv, 0, 128, None)
                                                                        for name, _, lens, new, _, Hq, Hkv, _ in TOGETHER])
def test_queries_that_are_not_numbers(name, lens, new, Hq, Hkv, latent, d, slots):
    """A row whose every logit is NaN gives NaN, for its lse too, on every path: it is not one that sees nothing."""
    def edit(ks, vs, q):
        q[::3, 0, 5] = np.nan
    c = Paged(len(lens) + Hq + 1, lens, new, Hq, Hkv, d, 64, latent=latent, tree=max(new) <= 64, edit=edit,
              pitch=None if slots is None else slots // 64)
    out, lse = c.buffers()
    c.call(out=out, lse=lse)
    c.check(out, lse)
    assert torch.isnan(lse[:c.T:3, 0]).all() and torch.isnan(out[:c.T:3, 0]).all()
    rest = torch.ones(c.T, Hq, dtype=torch.bool, device=DEV)
    rest[::3, 0] = False
    assert torch.isfinite(lse[:c.T][rest]).all() and torch.isfinite(out[:c.T][rest]).all()


def test_prefill_of_queries_that_are_not_numbers():
    from tests.test_gpu_attn import expand_case, expand_run

    def edit(q, kv, kr):
        q[::3, 0, 70] = float("nan")
    for d in (64, 128):
        c = expand_case(21, [300, 1, 130], [0, 10, 200], 2, d, edit=edit)
        _, lse = expand_run(c)
        assert torch.isnan(lse[:c["T"]:3, 0]).all() and torch.isfinite(lse[:c["T"], 1]).all()


@pytest.mark.parametrize("latent", [0, 512])
def test_empty_contexts_on_clusters(latent):
    """Fewer tiles than CTAs of a cluster, requests without tokens or pages, in tables that ask for clusters of eight."""
    c = Paged(3, [1, 0, 130, 40], [1, 0, 2, 5], 8, 2 if not latent else 1, 128, 64, latent=latent, pitch=15, missing=[(3, 0)])
    assert path(c.p, latent) == "cluster 8"
    out, lse = c.buffers()
    c.call(out=out, lse=lse)
    c.check(out, lse)
    assert not out[3:8].any() and torch.isneginf(lse[3:8]).all()


@pytest.mark.parametrize("latent", [0, 512])
def test_idle_ctas_of_clusters_again_and_again(latent):
    """Clusters of eight of which one CTA has the only tile, the others nothing to wait for before the join, in launches that follow
    each other closely."""
    lens = [1, 130, 40, 128, 5, 70, 129, 30] if latent else [1, 130, 40, 128]
    c = Paged(18, lens, [1] * len(lens), 8, 2 if not latent else 1, 128, 64, latent=latent, pitch=15)
    assert path(c.p, latent) == "cluster 8"
    first, first_lse = c.buffers()
    c.call(out=first, lse=first_lse)
    c.check(first, first_lse)
    made = [c.buffers() for _ in range(100)]
    st = new_status()
    for out, lse in made:
        c.call(out=out, lse=lse, status=st)
    ok(st)
    for out, lse in made:
        assert torch.equal(out[:c.T], first[:c.T]) and torch.equal(lse[:c.T], first_lse[:c.T])


# ---------------------------------------------------------------------------------------------------------------
# waits that run out
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("name", ["whole", "cluster 8", "list, by item, wide", "list, by cta"])
def test_waits_that_run_out(name):
    """No copy is issued: the kernel ends within its budget and says so, and the next call is right."""
    entry = next(e for e in PATHS if e[0] == name and (name != "list, by item, wide" or e[5]))
    _, lens, new, Hq, Hkv, latent, d, _ = entry
    c = Paged(7, lens, new, Hq, Hkv, d, 64, latent=latent, tree=True)
    assert path(c.p, latent) == name
    c.call()
    torch.cuda.synchronize()
    stalled = C.CosaAttnParams.from_buffer_copy(c.p)
    stalled.flags |= C.COSA_ATTN_FLAG_TEST_STALL
    st, t0 = new_status(), time.time()
    c.call(p=stalled, status=st)
    torch.cuda.synchronize()
    assert int(st) == -4 and 1.5 < time.time() - t0 < 9
    out, lse = c.buffers()
    st = new_status()
    c.call(out=out, lse=lse, status=st)
    ok(st)
    c.check(out, lse)


def test_prefill_waits_that_run_out():
    from tests.test_gpu_attn import expand_case, expand_run
    c = expand_case(3, [300, 90], [0, 10], 3, 128)
    expand_run(c)
    c["p"].flags |= C.COSA_ATTN_FLAG_TEST_STALL
    st, t0 = new_status(), time.time()
    C.cosa_latent_prefill(c["p"], *c["args"], cu_kv=c["cu_kv"], status=st)
    torch.cuda.synchronize()
    assert int(st) == -4 and 1.5 < time.time() - t0 < 9
    c["p"].flags = 0
    expand_run(c)


@pytest.mark.parametrize("form", ["prefill", "clusters"])
def test_ctas_that_start_after_a_timeout_end_at_once(form):
    """More CTAs than run at a time: one wait's time for all of them, not for each wave."""
    if form == "prefill":
        from tests.test_gpu_attn import expand_case, expand_run
        c = expand_case(4, [128 * 40, 128 * 30], [0, 10], 9, 64)       # 630 CTAs, one to an SM
        p, args = c["p"], c["args"]
        def call(**kw):
            C.cosa_latent_prefill(p, *args, cu_kv=c["cu_kv"], **kw)
    else:
        c = Paged(7, [1000] * 15, [1] * 15, 4, 1, 128, 64)
        assert path(c.p, 0) == "cluster 8"                             # 19 clusters, as many as 152 SMs would hold
        p, call = c.p, c.call
    call()
    torch.cuda.synchronize()
    p.flags |= C.COSA_ATTN_FLAG_TEST_STALL
    st, t0 = new_status(), time.time()
    call(status=st)
    torch.cuda.synchronize()
    assert int(st) == -4 and 1.5 < time.time() - t0 < 3.5
    p.flags = 0
    if form == "prefill":
        expand_run(c, check=False)
    else:
        out, lse = c.buffers()
        c.call(out=out, lse=lse)
        c.check(out, lse)


@pytest.mark.parametrize("name", ["whole", "cluster 8", "list, by item, wide", "list, by item", "list, by cta"])
def test_calls_after_a_timeout_touch_nothing_else(name):
    """A status that still says so: no CTA works, in workspaces of any content, and nothing but the outputs' rows is written."""
    for _, lens, new, Hq, Hkv, latent, d, slots in (e for e in PATHS if e[0] == name):
        c = Paged(8, lens, new, Hq, Hkv, d, 64, latent=latent, tree=True, pitch=None if slots is None else slots // 64)
        assert path(c.p, latent) == name
        size = (C.cosa_latent_attention_workspace_size if latent else C.cosa_tree_attention_workspace_size)(c.p)
        for fill in (0x00, 0x7F, 0xFF):
            ws = torch.full((size + 4096,), fill, dtype=torch.uint8, device=DEV)
            out, lse = c.buffers()
            guard, st, t0 = out.clone(), new_status(), time.time()
            st.fill_(-4)
            c.call(out=out, lse=lse, workspace=ws[:size], status=st)
            torch.cuda.synchronize()
            assert int(st) == -4 and time.time() - t0 < 1.5
            assert torch.equal(out[c.T:], guard[c.T:]) and (ws[size:] == fill).all()
            st = new_status()
            c.call(out=out, lse=lse, workspace=ws[:size], status=st)
            ok(st)
            c.check(out, lse)


# ---------------------------------------------------------------------------------------------------------------
# a step with drafted tokens: norm and rotation, tree attention, commit, and the next step over what was kept
# ---------------------------------------------------------------------------------------------------------------
def test_drafted_steps():
    rng = np.random.default_rng(11)
    B, Hq, Hkv, d, P, most = 3, 8, 2, 128, 16, 40
    pages = 12
    total = B * pages + 2
    t = table(rng, B, pages, total)
    kc, vc = (bf(rng, total, P, Hkv, d) for _ in range(2))
    length = np.array([60, 0, 17])
    inv = torch.from_numpy(1e4 ** (-np.arange(d // 2) / (d // 2))).to(DEV)
    w = [bf(rng, d) * 0.2 + 1 for _ in range(2)]
    kv_len = i32(length)
    # what each request keeps, in the reference
    hist = []
    for b in range(B):
        at = np.arange(length[b])
        phys = t[b][at // P]
        hist.append([to_f64(x)[phys, at % P] for x in (kc, vc)])
    for step in range(3):
        new = [13, 7, 20] if step < 2 else [1, 1, 1]
        masks = [[1] if n == 1 else None for n in new]
        up = [[-1] + [int(rng.integers(-1, i)) for i in range(1, n)] for n in new]
        depth = []
        for b, n in enumerate(new):
            m, dep = [], []
            for i, u in enumerate(up[b]):
                m.append((m[u] if u >= 0 else 0) | 1 << i)
                dep.append(dep[u] + 1 if u >= 0 else 0)
            masks[b] = m
            depth += [length[b] + x for x in dep]
        T = sum(new)
        qkv = bf(rng, T, Hq + 2 * Hkv, d)
        cu, start = cu_of(new), kv_len.clone()
        kv_len = kv_len + i32(new)
        kp = K.make_kv_params(num_reqs=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, page_size=P, total_tokens=T, max_seqlen=pages * P,
                              num_pages=total, max_pages_per_req=pages)
        st = new_status()
        q_out, _ = K.cosa_qk_norm_rope(kp, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], cu, inv, v=qkv[:, Hq + Hkv:], q_weight=w[0], k_weight=w[1],
                                       positions=i32(depth), start=start, k_cache=kc, v_cache=vc, page_table=i32(t), status=st)
        p = C.make_attn_params(num_reqs=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, page_size=P, total_tokens=T, max_seqlen=pages * P,
                               num_pages=total, max_pages_per_req=pages, max_new_tokens=most)
        lse = torch.empty(T, Hq, device=DEV)
        out = C.cosa_tree_attention(p, q_out, cu, kc, vc, i32(t), kv_len, tree_mask=bits(masks), lse=lse, status=st)
        paths = [[j for j in range(n) if masks[b][n - 1] >> j & 1] for b, n in enumerate(new)]
        kv_len = C.cosa_tree_commit(p, (kc, vc), cu, i32(t), kv_len, i32([x + [0] * (most - len(x)) for x in paths]), i32([len(x) for x in paths]),
                                    status=st)
        ok(st)
        # the cache's bf16 values come from the rotation, which other tests check
        rows, _ = norm_rope(to_f64(qkv[:, Hq:Hq + Hkv]), to_f64(w[1]), np.array(depth), inv.cpu().numpy(), False, 1e-6)
        at = 0
        for b, n in enumerate(new):
            L = length[b]
            k = np.concatenate([hist[b][0], np.zeros((n, Hkv, d))])
            v = np.concatenate([hist[b][1], to_f64(qkv[at:at + n, Hq + Hkv:])])
            k[L:] = bf16(rows[at:at + n])
            seen = ref.seen_of(L + n, n, masks[b])
            want = ref.attention(to_f64(q_out[at:at + n]), k, v, seen, p.sm_scale)
            # a rounding of a key that falls on the other side moves logits by 2^-8 of one product; keys are compared below
            near(to_f64(out[at:at + n]), to_f64(lse[at:at + n]), *want[:3], want[3] + 2.0 ** -9 * np.abs(want[1]).max(), L + n)
            keep = [L + j for j in paths[b]]
            length[b] = L + len(keep)
            hist[b] = [np.concatenate([k[:L], k[keep]]), np.concatenate([v[:L], v[keep]])]
            slots = np.arange(length[b])
            phys = t[b][slots // P]
            got_k, got_v = to_f64(kc)[phys, slots % P], to_f64(vc)[phys, slots % P]
            assert np.array_equal(got_v, hist[b][1])
            assert (np.abs(got_k - hist[b][0]) <= np.abs(hist[b][0]) * 2.0 ** -7 + 2.0 ** -14).all()
            hist[b][0] = got_k
            at += n
        assert kv_len.tolist() == length.tolist()


def test_latent_prompt_and_steps():
    """A prompt in the expanded form, then new tokens in the absorbed form over the pages that the prompt wrote: both against the
    definition with the same weights."""
    rng = np.random.default_rng(12)
    B, H, d, DL, P, pages = 2, 4, 128, 256, 32, 8
    lens = [150, 70]
    T = sum(lens)
    wk, wv = (bf(rng, H, DL, d) * DL ** -0.5 for _ in range(2))
    norm = bf(rng, DL) * 0.2 + 1
    inv = torch.from_numpy(1e4 ** (-np.arange(32) / 32)).to(DEV)
    t = table(rng, B, pages, B * pages)
    cache = torch.zeros(C.latent_cache_shape(B * pages, P, DL), dtype=torch.bfloat16, device=DEV)
    base = dict(num_reqs=B, num_q_heads=H, head_dim=d, latent_dim=DL, page_size=P, max_seqlen=pages * P, num_pages=B * pages, max_pages_per_req=pages,
                sm_scale=(d + 64) ** -0.5)
    p = C.make_attn_params(total_tokens=T, total_kv_tokens=T, max_new_tokens=150, **base)
    kv, q = bf(rng, T, DL + 64), bf(rng, T, H, d + 64)
    st = new_status()
    q_rope, c, k_rope = C.cosa_latent_rope(p, kv, cu_of(lens), inv, q=q[..., d:], weight=norm, c_out=torch.empty(T, DL, dtype=torch.bfloat16, device=DEV),
                                           k_out=torch.empty(T, 64, dtype=torch.bfloat16, device=DEV), cache=cache, page_table=i32(t), status=st)
    kk, vv = (torch.einsum("tc,hcd->thd", c.float(), x.float()).to(torch.bfloat16) for x in (wk, wv))
    out = C.cosa_latent_prefill(p, q[..., :d], q_rope, kk, k_rope, vv, cu_of(lens), status=st)
    ok(st)
    at = 0
    for b, n in enumerate(lens):
        s = slice(at, at + n)
        k = np.concatenate([to_f64(kk[s]), np.repeat(to_f64(k_rope[s])[:, None], H, 1)], -1)
        want = ref.attention(np.concatenate([to_f64(q[s, :, :d]), to_f64(q_rope[s])], -1), k, to_f64(vv[s]), np.tril(np.ones((n, n), bool)), p.sm_scale)
        near(to_f64(out[s]), None, *want, n)
        slots = np.arange(n)
        rows = to_f64(cache)[t[b][slots // P], slots % P]
        assert np.array_equal(rows[:, :DL], to_f64(c[s])) and np.array_equal(rows[:, DL:], to_f64(k_rope[s]))
        at += n
    # one more token each, absorbed
    length = np.array(lens)
    p1 = C.make_attn_params(total_tokens=B, **base)
    kv, q = bf(rng, B, DL + 64), bf(rng, B, H, d + 64)
    q_rope, _, _ = C.cosa_latent_rope(p1, kv, cu_of([1, 1]), inv, q=q[..., d:], weight=norm, start=i32(length), cache=cache, page_table=i32(t), status=st)
    q_latent = torch.einsum("thd,hcd->thc", q[..., :d].float(), wk.float()).to(torch.bfloat16)
    o = C.cosa_latent_attention(p1, q_latent, q_rope, cu_of([1, 1]), cache, i32(t), i32(length + 1), status=st)
    ok(st)
    for b in range(B):
        slots = np.arange(length[b] + 1)
        rows = to_f64(cache)[t[b][slots // P], slots % P][:, None]
        want = ref.attention(np.concatenate([to_f64(q_latent[b:b + 1]), to_f64(q_rope[b:b + 1])], -1), rows, rows[..., :DL],
                             np.ones((1, length[b] + 1), bool), p1.sm_scale)
        near(to_f64(o[b:b + 1]), None, *want, length[b] + 1)


# ---------------------------------------------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("latent", [0, 512])
@pytest.mark.parametrize("lens", [[300, 90], [9000, 4000]])
def test_two_streams_at_once(latent, lens):
    """Calls on two streams with their own workspaces, many times."""
    cs = [Paged(s, lens, [3, 2], 8, 2 if not latent else 1, 128, 64, latent=latent, tree=True) for s in (1, 2)]
    outs, streams = [c.buffers() for c in cs], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(8):
        for c, (out, lse), s in zip(cs, outs, streams):
            c.call(out=out, lse=lse, stream=s)
    torch.cuda.synchronize()
    for c, (out, lse) in zip(cs, outs):
        c.check(out, lse)


@pytest.mark.parametrize("latent", [0, 512])
@pytest.mark.parametrize("lens", [[300, 90], [9000, 4000]])
def test_graphs_that_share_nothing(latent, lens):
    """Two captured calls with other kernels around them, replayed at once, after new inputs were copied in."""
    cs = [Paged(s, lens, [3, 2], 8, 2 if not latent else 1, 128, 64, latent=latent, tree=True) for s in (3, 4)]
    size = C.cosa_latent_attention_workspace_size if latent else C.cosa_tree_attention_workspace_size
    made = []
    for c in cs:
        ws = torch.empty(size(c.p), dtype=torch.uint8, device=DEV)
        out, lse = c.buffers()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.call(out=out, lse=lse, workspace=ws)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out.zero_()
            c.call(out=out, lse=lse, workspace=ws)
            twice = out + out
        made.append((g, s, out, lse, twice, ws))
    for c, other in zip(cs, cs[::-1]):          # each graph's queries become the other's, negated, and its lengths shorter
        c.qf = -c.qf
        c.q.neg_()
        if c.q_rope is not None:
            c.q_rope.neg_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s, *_ in made:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (_, _, out, lse, twice, _) in zip(cs, made):
        c.check(out, lse)
        assert torch.equal(twice[:c.T], (out + out)[:c.T])


def test_graph_of_a_whole_step():
    """Norm and rotation, attention and commit in one graph, replayed after the lengths and the cache moved on."""
    rng = np.random.default_rng(5)
    B, H, DL, P, pages, n = 2, 16, 512, 16, 30, 4
    cache = bf(rng, B * pages, P, DL + 64)
    t = i32(table(rng, B, pages, B * pages))
    inv = torch.from_numpy(1e4 ** (-np.arange(32) / 32)).to(DEV)
    p = C.make_attn_params(num_reqs=B, num_q_heads=H, latent_dim=DL, page_size=P, total_tokens=B * n, max_seqlen=pages * P, num_pages=B * pages,
                           max_pages_per_req=pages, max_new_tokens=n, sm_scale=0.05)
    kv, q, ql = bf(rng, B * n, DL + 64), bf(rng, B * n, H, 64), bf(rng, B * n, H, DL)
    length, cu = i32([100, 37]), cu_of([n] * B)
    mask, path_, path_len = bits([[1, 3, 5, 11]] * B), i32([[0, 2, 0, 0], [0, 1, 3, 0]]), i32([2, 3])
    q_rope, out, after = torch.empty_like(q), torch.empty_like(ql), torch.empty(B, dtype=torch.int32, device=DEV)
    ws, st = torch.empty(C.cosa_latent_attention_workspace_size(p), dtype=torch.uint8, device=DEV), new_status()

    def step():
        C.cosa_latent_rope(p, kv, cu, inv, q=q, start=length, q_out=q_rope, cache=cache, page_table=t, status=st)
        full = length + n
        C.cosa_latent_attention(p, ql, q_rope, cu, cache, t, full, tree_mask=mask, out=out, workspace=ws, status=st)
        C.cosa_tree_commit(p, (cache,), cu, t, full, path_, path_len, new_len=after, status=st)
        length.copy_(after)

    before = cache.clone(), length.clone()
    eager = []
    for _ in range(4):
        step()
        eager.append((out.clone(), length.clone()))
    end = cache.clone()
    cache.copy_(before[0])
    length.copy_(before[1])
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        step()
    for o, m in eager:
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(length, m)
    assert torch.equal(cache, end) and length.tolist() == [108, 49]
    ok(st)


def test_memory_of_a_stream():
    """Outputs and workspace that a call on a stream allocates belong to that stream."""
    c = Paged(6, [2000, 90], [3, 2], 8, 2, 64, 32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = []
    for _ in range(4):
        out = c.call(stream=s)
        with torch.cuda.stream(s):
            junk = torch.full((1 << 22,), -1, dtype=torch.int32, device=DEV)     # would take a freed workspace on that stream
            kept.append(out)
        del junk
    torch.cuda.synchronize()
    for out in kept:
        c.check(out, None)


# ---------------------------------------------------------------------------------------------------------------
# large caches
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("latent", [0, 512])
def test_caches_beyond_32_bits(latent):
    """Pages whose bytes and elements are numbered beyond 2^32."""
    c = Paged(8, [700, 130], [3, 2], 8, 8 if not latent else 1, 128, 64, latent=latent, tree=True)
    far = 70000 if latent else 34000                       # pages: of 64 * 576 and 64 * 8 * 128 elements
    at = np.arange(c.total) * (far // c.total - 1) + far - (c.total - 1) * (far // c.total - 1) - 1

    def spread(cache):
        big = torch.empty((far, *cache.shape[1:]), dtype=cache.dtype, device=DEV)
        big[torch.from_numpy(at).to(DEV)] = cache
        assert big.numel() > 2 ** 31 if latent else big.numel() * 2 > 2 ** 32
        return big

    if latent:
        c.cache = spread(c.cache)
    else:
        c.k, c.v = spread(c.k), spread(c.v)
    c.t = at[c.t]
    c.pt, c.total = i32(c.t), far
    c.p.num_pages = far
    out, lse = c.buffers()
    st = new_status()
    c.call(out=out, lse=lse, status=st)
    ok(st)
    c.check(out, lse)
