"""The calls of include/cosa_kv.h on the paths that small shapes do not reach: the attention's list of the whole batch with its
join, whichever way its waits end, long contexts, many rows."""
import time

import numpy as np
import pytest
import torch

from block_sparse_long_gb300 import cosa, kv as C
from tests import kv_bulk, kv_paths, kv_reference as ref, test_gpu_kv as base, test_gpu_kv_serving as serving
from tests.kv_helpers import bf, cu_of, i32, new_status, ok

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_long_gb300 import build
    build.build()


# ---------------------------------------------------------------------------------------------------------------
# waits that run out
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 1), (24, 1), (30, 1)])
def test_waits_that_run_out_take_four_seconds_at_most(Hq, Hkv, listed):
    """Nothing is copied, so the first wait of every warp runs out, 2 s after it began; no copy is in flight to be waited for.
    The requests have one unit to four, so that in a list the warps of a CTA come to their first wait in different items."""
    lens = [10, 30, 50, 70, 20, 100, 128, 1, 15]
    c = base.attend(np.random.default_rng(Hq), lens, [1] * len(lens), Hq, Hkv, 64, 16, spare=0)
    if listed:
        kv_paths.widened(c)
    assert kv_paths.shares_a_list(c["p"]) == listed
    out = base.run_attention(c).clone()
    p = C.CosaKvParams.from_buffer_copy(c["p"])
    p.flags |= C.COSA_KV_FLAG_TEST_STALL
    st = new_status()
    args = (c["q"], cu_of(c["new"]), c["cache"], i32(c["t"]), i32(c["lens"]))
    torch.cuda.synchronize()
    t0 = time.monotonic()
    C.cosa_kv4_attention(p, *args, status=st)
    torch.cuda.synchronize()
    took = time.monotonic() - t0
    assert int(st.item()) == cosa.COSA_ERR_DEVICE_TIMEOUT
    assert 1.9 < took < 4.0, took
    st = new_status()
    assert torch.equal(C.cosa_kv4_attention(c["p"], *args, status=st), out)      # and the next call is as good as ever
    ok(st)


# ---------------------------------------------------------------------------------------------------------------
# contradictions
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("listed", [False, True])
def test_attention_reports_rows_before_the_first_request(listed):
    """cu_seqlens that begin behind row 0: reported, the rows in front left as they were, the requests served."""
    c = base.attend(np.random.default_rng(41), [30, 50, 9], [1, 2, 1], 4, 2, 64, 16, spare=1)
    if listed:
        kv_paths.widened(c)
    assert kv_paths.shares_a_list(c["p"]) == listed
    want = base.run_attention(c)
    shifted = torch.cat([c["q"][-1:], c["q"][:-1]])
    st, out = new_status(), torch.full_like(shifted, 7.0)
    C.cosa_kv4_attention(c["p"], shifted, cu_of(c["new"]) + 1, c["cache"], i32(c["t"]), i32(c["lens"]), out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == cosa.COSA_ERR_BAD_INPUT
    assert (out[0] == 7).all() and torch.equal(out[1:], want[:-1])
    st = new_status()                                            # and where no request has a query
    C.cosa_kv4_attention(c["p"], shifted, i32([2, 2, 2, 2]), c["cache"], i32(c["t"]), i32(c["lens"]), out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == cosa.COSA_ERR_BAD_INPUT and torch.equal(out[1:], want[:-1])


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("cu,start,dropped,reported", [
    ([0, 4, 9], [0, 0], [], (True, True)),             # a row more than there are
    ([0, 4, 8], [0, 13], [7], (True, False)),          # slots 13 to 16 of 16: without caches a slot is only a position
    ([0, 4, 8], [-2, 0], [0, 1], (True, True)),        # slots from -2
    ([1, 4, 8], [0, 0], [0], (True, True))])           # a row of no request
def test_rope_leaves_out_the_tokens_that_do_not_fit(cu, start, dropped, reported, paged):
    """Contradictions are reported; the tokens concerned are left out, all others of the request are written."""
    c = base.rope_case(43, [4, 4], [0, 0], 4, 2, 64, 16, 64, False, spare_rows=0)
    total, rng = c["p"].num_pages, c["rng"]
    kc, vc = (base.bf(rng, total, 16, 2, 64) for _ in range(2))
    q_out, k_out = base.bf(rng, 8, 4, 64), base.bf(rng, 8, 2, 64)
    before = [x.clone() for x in (q_out, k_out, kc, vc)]
    more = dict(v=c["v"], k_cache=kc, v_cache=vc, page_table=i32(c["t"])) if paged else {}
    st = new_status()
    C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], i32(cu), c["inv"], q_weight=c["wq"], k_weight=c["wk"], start=i32(start), q_out=q_out,
                        k_out=k_out, status=st, **more)
    torch.cuda.synchronize()
    if not paged and not reported[1]:
        dropped = []
    assert int(st.item()) == (cosa.COSA_ERR_BAD_INPUT if reported[0 if paged else 1] else 0)
    slots = np.array([t - cu[int(t >= cu[1])] + start[int(t >= cu[1])] for t in range(8)])
    c["pos"] = np.maximum(slots, 0)
    (yq, mq), (yk, mk) = base.rope_want(c)
    kept = [t for t in range(8) if t not in dropped]
    base.near(q_out[kept], yq[kept], mq[kept] * 2.0 ** -16)
    base.near(k_out[kept], yk[kept], mk[kept] * 2.0 ** -16)
    assert torch.equal(q_out[dropped], before[0][dropped]) and torch.equal(k_out[dropped], before[1][dropped])
    want_k, want_v = before[2], before[3]
    if paged:
        for t in kept:
            page = int(c["t"][int(t >= cu[1]), 0])
            want_k[page, slots[t]], want_v[page, slots[t]] = k_out[t], c["v"][t]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


# ---------------------------------------------------------------------------------------------------------------
# the list of the whole batch and its join
# ---------------------------------------------------------------------------------------------------------------
def attend_listed(rng, lens, new, Hq, Hkv, d, P, *, weights=False, missing=(), edit=None, hint=None, scale=None, q_scale=1.5, spare=2):
    """A case for base.run_attention whose batch is shared as one list."""
    cache, t, ks, vs = kv_bulk.packed(rng, lens, Hkv, P, d, missing=missing, edit=edit)
    T, pages = sum(new), t.shape[1]
    p = C.make_kv_params(num_reqs=len(lens), num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, page_size=P, total_tokens=T + spare,
                         max_seqlen=pages * P, num_kv4_pages=cache.shape[0], max_pages_per_req=pages,
                         max_new_tokens=max(1, max(new)) if hint is None else hint, sm_scale=scale)
    acc = torch.from_numpy(rng.random((len(lens), Hkv, pages * P)).astype(np.float32)).to(DEV) if weights else None
    c = dict(p=p, q=bf(rng, T + spare, Hq, d, scale=q_scale), cache=cache, t=t, ks=ks, vs=vs, lens=lens, new=new, acc=acc, T=T, P=P, rng=rng)
    return kv_paths.widened(c, max(40000, max(lens)))


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,P", [(32, 8, 128, 64), (4, 4, 64, 16), (7, 1, 128, 128), (8, 1, 64, 64), (12, 4, 128, 32), (9, 3, 64, 128),
                                        (16, 1, 128, 16), (16, 1, 64, 32), (9, 1, 64, 128), (24, 1, 64, 32), (20, 1, 128, 32),
                                        (24, 1, 128, 128), (33, 1, 128, 64), (40, 1, 64, 16)])
def test_listed_lengths(Hq, Hkv, d, P, weights):
    """One token per request; lengths from zero to several tiles; pages that end inside the tile; missing pages."""
    lens = [1, 15, 16, 17, 0, 64, 130, 300, 2, P + 1]
    base.run_attention(attend_listed(np.random.default_rng(Hq * 7 + d + P), lens, [1] * len(lens), Hq, Hkv, d, P, weights=weights,
                                     missing=[(7, 0), (6, min(1, 130 // P)), (2, 0)]))


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,new,hint", [(8, 2, 128, [3, 0, 1, 5, 2], None), (8, 2, 128, [3, 0, 1, 5, 2], 1), (4, 4, 64, [9, 1, 0, 20, 2], None),
                                               (16, 2, 64, [2, 0, 1, 3, 2], 2), (6, 2, 128, [40, 0, 1, 2, 2], 100), (5, 5, 128, [8, 8, 8, 8, 2], 3),
                                               (7, 1, 64, [3, 1, 1, 2, 0], None), (6, 1, 128, [4, 0, 1, 8, 1], None), (12, 1, 128, [2, 2, 2, 2, 2], 1)])
def test_listed_several_tokens(Hq, Hkv, d, new, hint, weights):
    """Causal at the end; several row tiles; requests without queries; queries that see nothing; hints too small and too large."""
    base.run_attention(attend_listed(np.random.default_rng(sum(new) + d), [100, 50, 1, 7, 1], new, Hq, Hkv, d, 16, weights=weights, hint=hint))


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,lens,new", [
    (32, 8, 64, [3000, 1, 0, 700, 33, 2048, 5, 900, 260], 1), (16, 8, 128, [1500, 64, 1, 31, 32, 700, 0, 90, 400, 17], 1),
    (36, 4, 64, [2000 - 111 * b for b in range(17)], 1), (20, 4, 64, [1200 - 60 * b for b in range(18)], 4),
    (8, 8, 128, [5] * 70, 1)])
def test_listed_many_items(Hq, Hkv, d, lens, new, weights):
    """More than 64 items: the join with a warp per row; CTAs' runs end inside items and span them."""
    c = attend_listed(np.random.default_rng(len(lens) + d), lens, [min(new, n) for n in lens], Hq, Hkv, d, 64, weights=weights,
                      missing=[(0, 3)] if max(lens) > 256 else [])
    assert kv_paths.items(c["p"]) > 64
    base.run_attention(c)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,lens", [(4, 1, 64, [25001]), (8, 1, 128, [12001]), (5, 1, 64, [70001]), (12, 1, 64, [40007]),
                                           (20, 1, 128, [12345]), (6, 2, 128, [31000, 4])])
def test_listed_long_contexts(Hq, Hkv, d, lens, weights):
    """Few items of very many parts: a thread of the join has more parts of a row than it asks for at once (128 of them for heads of
    64, 64 for 128)."""
    c = attend_listed(np.random.default_rng(lens[0]), lens, [1] * len(lens), Hq, Hkv, d, 128, weights=weights, missing=[(0, 2), (0, 40)])
    assert kv_paths.items(c["p"]) <= 64 and kv_paths.parts_of_the_longest(c["p"], lens) > (128 if d == 64 else 64)
    base.run_attention(c)


def test_listed_any_hint():
    c = attend_listed(np.random.default_rng(23), [700, 3, 90], [2, 0, 3], 8, 2, 128, 16, weights=True, hint=7)
    acc0, out = c["acc"].clone(), base.run_attention(c)
    acc1, c["acc"], c["p"].max_new_tokens, c["rng"] = c["acc"], acc0, 2 ** 31 - 1, np.random.default_rng(24)
    assert kv_paths.shares_a_list(c["p"])
    assert torch.equal(base.run_attention(c)[:c["T"]], out[:c["T"]]) and torch.equal(c["acc"], acc1)


def test_listed_large_logits_and_scale():
    """A maximum that moves late by hundreds, within a CTA's part and from part to part."""
    def edit(b, k, v):
        for s in range(0, len(k), 97):
            k[s] = ref.bf16(k[s] * (1 + s / 100))
    base.run_attention(attend_listed(np.random.default_rng(11), [1700, 190], [1, 2], 4, 2, 128, 16, weights=True, edit=edit, scale=0.02, q_scale=4.0))


def test_listed_keeps_nan_where_it_is_seen():
    """A NaN group of a key, of a value, in one part of many: rows that see the slot give NaN (for a value, in its 32
    channels), the others do not."""
    def edit(b, k, v):
        if b == 0:
            k[1010, 0, 3] = np.nan
        if b == 1:
            v[1499, 1, 40] = np.inf
    c = attend_listed(np.random.default_rng(12), [1500, 1500, 1500], [1, 2, 1], 4, 2, 64, 16, edit=edit)
    out = torch.zeros_like(c["q"])
    C.cosa_kv4_attention(c["p"], c["q"], cu_of(c["new"]), c["cache"], i32(c["t"]), i32(c["lens"]), out=out)
    o = ref.to_f64(out)
    assert np.isnan(o[0, :2]).all() and np.isfinite(o[0, 2:]).all()
    assert np.isfinite(o[1]).all()                                               # request 1's first token does not see slot 1499
    assert np.isfinite(o[2, :2]).all() and np.isfinite(o[2, 2:, :32]).all() and np.isnan(o[2, 2:, 32:]).all()
    assert np.isfinite(o[3]).all()


def test_listed_reports_contradictions():
    """The request concerned is empty (its rows stay as they were), the others are served; by other CTAs than without it, which
    may round differently: the reference decides."""
    c = attend_listed(np.random.default_rng(13), [900, 30, 700], [1, 1, 1], 2, 1, 64, 16, spare=0)
    top, q = c["p"].max_seqlen, ref.to_f64(c["q"])
    for cu, lens, served in (([0, 1, 2, 3], [900, top + 1, 700], (0, 2)), ([0, 1, 2, 3], [900, -1, 700], (0, 2)),
                             ([0, 1, 2, 4], [900, 30, 700], (0, 1)), ([0, 1, 4, 3], [900, 30, 700], (0,))):
        st, out = new_status(), torch.full_like(c["q"], 7.0)
        C.cosa_kv4_attention(c["p"], c["q"], i32(cu), c["cache"], i32(c["t"]), i32(lens), out=out, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == cosa.COSA_ERR_BAD_INPUT
        for b in range(3):
            if b not in served:
                assert (out[b] == 7).all()
                continue
            k, v = c["ks"][b], c["vs"][b]
            want, mag, _ = ref.attention(q[b:b + 1], k, v, np.ones(len(k), bool), c["p"].sm_scale)
            base.near(out[b:b + 1], want, mag * (2.0 ** -8 + 2.0 ** -17 + 2.1 * ref.logit_error(q[b:b + 1], k, c["p"].sm_scale)))


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("lens", [[900, 40, 333], [200 + 37 * b for b in range(20)]])
def test_listed_whatever_the_workspace_holds(lens, weights):
    """Owners and parts lie in the workspace: its content on entry, NaN and an earlier call's among them, changes nothing."""
    new = [1 + b % 2 for b in range(len(lens))]
    c = attend_listed(np.random.default_rng(14), lens, new, 8, 4, 128, 64, weights=weights)
    ws = torch.empty(C.cosa_kv4_attention_workspace_size(c["p"], weights), dtype=torch.uint8, device=DEV)
    args, acc0, outs = (c["p"], c["q"], cu_of(new), c["cache"], i32(c["t"]), i32(lens)), c["acc"], []
    for fill in (0, 255, 127, 7, None):                                          # None: as the call before it left it
        if fill is not None:
            ws.fill_(fill)
        acc = acc0.clone() if weights else None
        outs.append((C.cosa_kv4_attention(*args, weights=acc, workspace=ws)[:c["T"]].clone(), acc))
    for o, a in outs[1:]:
        assert torch.equal(o, outs[0][0]) and (not weights or torch.equal(a, outs[0][1]))


# ---------------------------------------------------------------------------------------------------------------
# many tokens into the cache and back
# ---------------------------------------------------------------------------------------------------------------
def placed(t, lens, starts, P, total):
    """(physical page, row, token) of the tokens whose pages exist, requests after each other."""
    b = np.repeat(np.arange(len(lens)), lens)
    slot = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, lens)])
    phys = t[b, slot // P].astype(np.int64)
    there = np.nonzero((phys >= 0) & (phys < total))[0]
    return phys[there], (slot % P)[there], there


@pytest.mark.parametrize("H,d,P", [(8, 128, 64), (9, 64, 16), (2, 64, 32), (3, 128, 128), (1, 64, 128), (12, 128, 16)])
def test_bulk_rows(H, d, P):
    """More rows than go one to a CTA: CTAs of 8 or 16 tokens that cross requests (some of them empty) and pages, a last CTA with
    fewer, rows behind the last request."""
    rng = np.random.default_rng(H + d + P)
    lens, starts = [1, 0, 5, 1013, 0, 0, 2, 1, 1, 1, 700, 3, 0, 411, 9], [0, 4, P - 2, 7, 1, 0, 2 * P + 1, 3, 3, 0, P, 1, 0, 15, 16]
    T, pages = sum(lens), max(-(-(s + n) // P) for s, n in zip(starts, lens))
    assert T % 16 and T % 8 and T > 8 * 152
    kv = base.bf(rng, T + 3, 2 * H * d + 8)
    k, v = kv[:, :H * d].unflatten(1, (H, d)), kv[:, H * d:2 * H * d].unflatten(1, (H, d))
    base.special(rng, k[30:])
    base.special(rng, v[900:])
    total = len(lens) * pages + 1
    t = base.table(rng, len(lens), pages, total, missing=[(3, 1), (10, 2), (6, 2)])
    cache = base.noise_cache(rng, total, H, P, d)
    want = cache.cpu().numpy().copy()
    p = C.make_kv_params(num_reqs=len(lens), num_q_heads=H, num_kv_heads=H, head_dim=d, page_size=P, total_tokens=T + 3,
                         max_seqlen=pages * P, num_kv4_pages=total, max_pages_per_req=pages)
    st = new_status()
    C.cosa_kv4_store(p, cache, i32(t), k, v, cu_seqlens=cu_of(lens), start=i32(starts), status=st)
    ok(st)
    phys, row, tok = placed(t, lens, starts, P, total)
    kv_bulk.put(want, phys, row, ref.to_f64(k)[tok], ref.to_f64(v)[tok])
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("H,d,P,B,long", [(8, 64, 64, 64, 1500), (2, 128, 128, 64, 3000), (3, 64, 16, 64, 4001), (1, 64, 16, 5000, 60), (9, 64, 32, 1, 45000)])
def test_pages_of_requests_longer_than_a_turn_of_their_CTAs(H, d, P, B, long):
    """A request's CTAs (4864 over the batch) take up to 16 slots each at a time and come round again: store and load, from a
    start inside a tile; pages without a counterpart on either side."""
    tokens, most = (8 if H >= 8 else 16), max(1, 32 * 152 // B)
    assert long - 37 > tokens * most
    rng = np.random.default_rng(H + d + P + B)
    ends = [long] + [int(n) for n in rng.integers(0, min(long, 40) + 1, B - 1)]
    starts = [37] + [int(n) for n in rng.integers(0, 20, B - 1)]
    lens = [max(0, e - s) for s, e in zip(starts, ends)]
    pages = -(-long // P)
    # the long request's pages, and one or three for each other: the rest of the tables points nowhere
    few = min(pages, -(-40 // P))
    total = pages + (B - 1) * few + 2
    def tables():
        perm = rng.permutation(total).astype(np.int32)
        t = np.full((B, pages), -1, np.int32)
        t[0], t[1:, :few] = perm[:pages], perm[pages:pages + (B - 1) * few].reshape(B - 1, few)
        t[0, int(rng.integers(1, pages))] = total + 5
        return t
    t4, t16 = tables(), tables()
    k, v = base.bf(rng, total, P, H, d), base.bf(rng, total, P, H, d)
    base.special(rng, k[:, 3])
    cache = base.noise_cache(rng, total, H, P, d)
    want = cache.cpu().numpy().copy()
    p = C.make_kv_params(num_reqs=B, num_q_heads=H, num_kv_heads=H, head_dim=d, page_size=P, max_seqlen=pages * P, num_pages=total,
                         num_kv4_pages=total, max_pages_per_req=pages)
    st = new_status()
    C.cosa_kv4_store(p, cache, i32(t4), k, v, src_page_table=i32(t16), start=i32(starts), kv_len=i32(ends), status=st)
    ok(st)
    b = np.repeat(np.arange(B), lens)
    slot = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, lens)])
    a, z = t16[b, slot // P].astype(np.int64), t4[b, slot // P].astype(np.int64)
    both = (a >= 0) & (a < total) & (z >= 0) & (z < total)
    a, z, row = a[both], z[both], (slot % P)[both]
    assert both.sum() > long // 2 and not both.all()
    kv_bulk.put(want, z, row, ref.to_f64(k)[a, row], ref.to_f64(v)[a, row])
    assert np.array_equal(cache.cpu().numpy(), want)

    # and back into other contents of the same pages
    kb, vb = base.bf(rng, total, P, H, d), base.bf(rng, total, P, H, d)
    want_k, want_v = ref.to_f64(kb), ref.to_f64(vb)
    C.cosa_kv4_load(p, cache, i32(t4), kb, vb, i32(t16), kv_len=i32(ends), start=i32(starts), status=st)
    ok(st)
    x, y = kv_bulk.get(want, z, row, d)
    want_k[a, row], want_v[a, row] = ref.bf16(x), ref.bf16(y)
    assert np.array_equal(ref.to_f64(kb), want_k, equal_nan=True) and np.array_equal(ref.to_f64(vb), want_v, equal_nan=True)


# ---------------------------------------------------------------------------------------------------------------
# memory that the binding allocates
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("which", ["rope", "attention", "attention with weights", "evict"])
def test_allocated_memory_belongs_to_the_streams_pool(monkeypatch, which):
    """What the binding allocates for a call on a given stream is that stream's memory: freed at once while the call still waits,
    none of it is handed out to the current stream."""
    c = attend_listed(np.random.default_rng(51), [700, 90], [1, 1], 8, 2, 64, 16, weights=which.endswith("weights"), spare=0)
    p, inv = c["p"], torch.from_numpy(1e4 ** (-np.arange(32) / 32)).to(DEV)
    p.budget, p.max_dst_pages = 16, 1
    cu, t, lens, k = cu_of([1, 1]), i32(c["t"]), i32(c["lens"]), bf(c["rng"], 2, 2, 64)
    room, few = i32(np.setdiff1d(np.arange(c["cache"].shape[0]), c["t"])[:2].reshape(2, 1)), i32([8, 9])
    w = torch.rand(2, 2, p.max_seqlen, device=DEV)
    call = {"rope": lambda st: C.cosa_qk_norm_rope(p, c["q"], k, cu, inv, stream=st),
            "evict": lambda st: C.cosa_kv4_evict(p, c["cache"], t, few, w, room, stream=st)}.get(
                which, lambda st: C.cosa_kv4_attention(p, c["q"], cu, c["cache"], t, lens, weights=c["acc"], stream=st))
    call(None)                                # loads the kernels
    blocks, empty = [], C._Call.empty

    def recorded(self, shape, dtype, stream):
        got = empty(self, shape, dtype, stream)
        blocks.append((got.data_ptr(), got.shape, got.dtype))
        return got

    monkeypatch.setattr(C._Call, "empty", recorded)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)        # the stream is busy: the call waits
    call(side)                                # what it returns is let go
    again = [torch.empty(shape, dtype=dtype, device=DEV) for _, shape, dtype in blocks for _ in range(3)]
    busy = not side.query()
    torch.cuda.synchronize()
    assert busy, "the stream ended too soon for the check to mean anything"
    assert len(blocks) == {"rope": 2, "evict": 3}.get(which, 2)
    assert not {a for a, _, _ in blocks} & {x.data_ptr() for x in again}


def test_evict_without_weights_out():
    """The C call makes weights_out optional: the same slots, kept numbers and moved rows without it."""
    rng = np.random.default_rng(61)
    cache, t, _, _ = kv_bulk.packed(rng, [300, 40], 2, 16, 64)
    pages, room = t.shape[1], 3
    dst = np.setdiff1d(np.arange(cache.shape[0] + 2 * room), t)[-2 * room:].reshape(2, room)
    cache = torch.cat([cache, torch.zeros_like(cache[:2 * room])])
    p = C.make_kv_params(num_reqs=2, num_q_heads=2, num_kv_heads=2, head_dim=64, page_size=16, max_seqlen=pages * 16, num_kv4_pages=cache.shape[0],
                         max_pages_per_req=pages, budget=40, sink=2, recent=5, max_dst_pages=room)
    w = torch.from_numpy(rng.exponential(size=(2, 2, pages * 16)).astype(np.float32)).to(DEV)
    table, lens, to = i32(t), i32([300, 40]), i32(dst)
    other = cache.clone()
    new_len, kept, _ = C.cosa_kv4_evict(p, cache, table, lens, w, to)
    n2, k2, st = torch.zeros_like(new_len), torch.zeros_like(kept), new_status()
    rc = C.kv_library().cosa_kv4_evict(p, other.data_ptr(), table.data_ptr(), lens.data_ptr(), w.data_ptr(), to.data_ptr(), n2.data_ptr(),
                                       k2.data_ptr(), None, st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    ok(st)
    assert torch.equal(n2, new_len) and torch.equal(k2, kept) and torch.equal(other, cache) and new_len.tolist() == [40, 40]


# ---------------------------------------------------------------------------------------------------------------
# calls of one program on two streams
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("listed", [False, True])
def test_decode_over_two_streams_and_captured(listed):
    """Norm and rotation on one stream, append and attention on another behind an event, torch's kernels and fills between them, the
    eviction back on the first: the results of one stream, run by run and replayed from a graph.  (Kernels of the library start
    before the one in front of them has ended, and wait.)"""
    s = serving.Loop(71)
    s.prefill()
    ok(s.status)
    B, d = 2, s.d
    pages = 2500 if listed else s.pages
    pt4 = np.full((B, pages), -1, np.int32)
    pt4[:, :s.pages] = s.pt4
    p1 = C.make_kv_params(total_tokens=B, **{**s.common, "max_seqlen": pages * s.P, "max_pages_per_req": pages})
    assert kv_paths.shares_a_list(p1) == listed
    table, dst, cu1, before, after = i32(pt4), i32(s.dst), cu_of([1] * B), i32(s.lens), i32([n + 1 for n in s.lens])
    pos, x, cache0 = i32(s.pos), s.steps[0], s.cache.clone()
    e = lambda *a, dtype=torch.bfloat16: torch.zeros(a, dtype=dtype, device=DEV)  # noqa: E731
    q1, k1, v1, out = e(B, s.Hq, d), e(B, s.Hkv, d), e(B, s.Hkv, d), e(B, s.Hq, d)
    acc, acc_out = (e(B, s.Hkv, pages * s.P, dtype=torch.float32) for _ in range(2))
    n, kept, ws = e(B, dtype=torch.int32), e(B, s.Hkv, s.budget, dtype=torch.int32), torch.empty(
        C.cosa_kv4_attention_workspace_size(p1, True), dtype=torch.uint8, device=DEV)
    outs = [q1, k1, out, acc, n, kept, acc_out, s.cache]

    def step(main, side):
        with torch.cuda.stream(main):
            s.cache.copy_(cache0)
            q, k, v = s.split(x)
            C.cosa_qk_norm_rope(p1, q, k, cu1, s.inv, q_weight=s.wq, k_weight=s.wk, positions=pos, q_out=q1, k_out=k1)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            acc.zero_()
            v1.copy_(v)
            C.cosa_kv4_store(p1, s.cache, table, k1, v1, cu_seqlens=cu1, start=before)
            C.cosa_kv4_attention(p1, q1, cu1, s.cache, table, after, out=out, weights=acc, workspace=ws)
            acc.mul_(0.5)
            C.cosa_kv4_attention(p1, q1, cu1, s.cache, table, after, out=out, weights=acc, workspace=ws)
        main.wait_stream(side)
        with torch.cuda.stream(main):
            C.cosa_kv4_evict(p1, s.cache, table, after, acc, dst, new_len=n, kept=kept, weights_out=acc_out)

    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    step(one, one)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    assert all(bool((t != 0).any()) for t in want)
    for _ in range(10):
        for t in outs[:-1]:
            t.zero_()
        torch.cuda.synchronize()
        step(one, two)
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=one):
        step(one, two)
    for _ in range(3):
        for t in outs[:-1]:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(outs, want))
