"""The calls of include/cosa_attn.h on the GPU against tests/attn_reference.py; the tolerances are derived there and in
tests/attn_helpers.near.  Caches hold NaN, infinities and large values wherever no slot is."""
import numpy as np
import pytest
import torch

from block_sparse_long_gb300 import attn as C
from tests import attn_reference as ref
from tests.attn_helpers import DEV, Paged, garbage, near, random_masks, there_of
from tests.kv_helpers import bf, cu_of, i32, new_status, ok, table
from tests.kv_reference import bf16, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_long_gb300 import build
    build.build()


def run_and_check(c, **kw):
    out, lse = c.buffers()
    guard, guard_lse, st = out.clone(), lse.clone(), new_status()
    got = c.call(out=out, lse=lse, status=st, **kw)
    ok(st)
    assert got is out
    c.check(out, lse)
    assert torch.equal(out[c.T:], guard[c.T:]) and torch.equal(lse[c.T:], guard_lse[c.T:])     # rows behind the last request
    return out, lse


# ---------------------------------------------------------------------------------------------------------------
# attention over pages
# ---------------------------------------------------------------------------------------------------------------
HEADS = [(32, 8, 128, 64), (4, 4, 64, 16), (7, 1, 128, 128), (8, 1, 64, 32), (3, 1, 128, 16), (64, 2, 128, 64), (6, 2, 64, 128), (1, 1, 64, 64)]


@pytest.mark.parametrize("Hq,Hkv,d,P", HEADS)
@pytest.mark.parametrize("tree", [False, True])
def test_tree_attention(Hq, Hkv, d, P, tree):
    c = Paged(Hq * 100 + d + P + tree, [1, 130, 0, 257, 64, 700, 33], [1, 3, 0, 5, 2, 13, 33], Hq, Hkv, d, P, tree=tree,
              missing=[(3, 1), (5, 2)] if P < 128 else [(5, 0)])
    run_and_check(c)


@pytest.mark.parametrize("H,latent,P", [(16, 512, 64), (32, 512, 16), (5, 512, 128), (1, 256, 32), (24, 256, 64), (128, 512, 64), (64, 256, 16)])
@pytest.mark.parametrize("tree", [False, True])
def test_latent_attention(H, latent, P, tree):
    c = Paged(H * 100 + latent + P + tree, [1, 130, 0, 257, 64, 500, 9], [1, 3, 0, 2, 4, 7, 9], H, latent=latent, P=P, tree=tree,
              missing=[(3, 1), (5, 2)] if P < 128 else [(5, 0)])
    run_and_check(c)


@pytest.mark.parametrize("latent", [0, 512])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 63, 64])
def test_tree_widths(latent, n):
    """Trees of every kind of width, the bits of the widest up to the sign, over contexts that end around a tile's border."""
    for ctx in (0, 1, 127 - min(n, 127) % 128, 128, 200):
        run_and_check(Paged(n * 7 + ctx, [ctx + n, 3 + n], [n, n], 4, 2 if not latent else 1, 64, 16, latent=latent, tree=True))


@pytest.mark.parametrize("latent", [0, 512])
def test_long_contexts_are_shared(latent):
    """Contexts that many CTAs share, beside short ones."""
    c = Paged(5, [9001, 1, 4000, 130], [4, 1, 2, 3], 8, 2 if not latent else 1, 128, 32, latent=latent, tree=True)
    run_and_check(c)


@pytest.mark.parametrize("latent,d", [(0, 64), (0, 128), (256, 128), (512, 128)])
@pytest.mark.parametrize("new", [1, 3, 7, 15])
def test_many_tiles_to_a_cta(latent, d, new):
    """Every width of row tiles (8 rows a token: 16 to 128), with tens of tiles and several items to a CTA."""
    heads = 8 if latent else 16
    c = Paged(new + d + latent, [9000, 30011, 140, 20000], [new, 1, min(new, 4), new], heads, 1 if latent else 2, d, 64, latent=latent, tree=True)
    for _ in range(3):
        out, lse = c.buffers()
        st = new_status()
        for _ in range(4):
            c.call(out=out, lse=lse, status=st)
        ok(st)
    c.check(out, lse)


@pytest.mark.parametrize("latent", [0, 256])
def test_many_requests(latent):
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 300, 300)]
    c = Paged(6, lens, [min(n, 1 + i % 3) for i, n in enumerate(lens)], 4, 2 if not latent else 1, 64, 32, latent=latent)
    run_and_check(c)


@pytest.mark.parametrize("latent", [0, 512])
def test_chain_longer_than_a_tree(latent):
    """Without masks any number of new tokens."""
    run_and_check(Paged(8, [300, 90], [150, 90], 4, 2 if not latent else 1, 128, 64, latent=latent))


@pytest.mark.parametrize("latent", [0, 512])
@pytest.mark.parametrize("strided", ["tokens", "heads"])
def test_tokens_and_heads_apart(latent, strided):
    run_and_check(Paged(9, [200, 77], [3, 2], 8, 2 if not latent else 1, 64, 32, latent=latent, strided=strided))


@pytest.mark.parametrize("latent", [0, 512])
@pytest.mark.parametrize("hint", [1, 2, 64, 1000])
def test_any_hint(latent, hint):
    c = Paged(10, [400, 60, 5], [9, 20, 1], 8, 2 if not latent else 1, 64, 32, latent=latent, tree=True)
    c.p.max_new_tokens = hint
    run_and_check(c)


@pytest.mark.parametrize("latent", [0, 512])
def test_rows_that_see_nothing(latent):
    """Masks without bits over no context, and a context without pages."""
    c = Paged(11, [9, 40, 12], [9, 5, 3], 4, 2 if not latent else 1, 64, 16, latent=latent, tree=True, ragged=True,
              missing=[(1, 0), (1, 1), (1, 2)])
    out, lse = run_and_check(c)
    assert not out[0].any() and torch.isneginf(lse[0]).all()            # the first mask has no bit
    assert not out[9:14].any() and torch.isneginf(lse[9:14]).all()


@pytest.mark.parametrize("latent", [0, 512])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_what_a_row_does_not_see_does_not_change_it(latent, bad):
    """One token of a tree has keys or values that are not finite: those that see it get what the definition gives, the others
    their result."""
    def edit(ks, vs, q):
        vs[0][205 - 6 + 2, 0, 3] = bad          # (latent: its key too)
        if not latent:
            ks[1][70 - 3 + 1, 0] = np.nan
    c = Paged(12, [205, 70], [6, 3], 4, 2 if not latent else 1, 64, 32, latent=latent, edit=edit)
    c.masks = [[1, 3, 4, 9, 20, 33], [1, 2, 5]]
    from tests.attn_helpers import bits
    c.mask = torch.cat([bits(c.masks), torch.zeros(3, dtype=torch.int64, device=DEV)])
    out, lse = c.buffers()
    c.call(out=out, lse=lse)
    got = to_f64(out)
    sees = [False, False, True, False, True, False]
    clean = Paged(12, [205, 70], [6, 3], 4, 2 if not latent else 1, 64, 32, latent=latent)
    clean.masks, clean.mask = c.masks, c.mask
    want, want_lse = clean.buffers()
    clean.call(out=want, lse=want_lse)
    for i, s in enumerate(sees):
        if not s:
            assert torch.equal(out[i], want[i]) and torch.equal(lse[i], want_lse[i]), i
        else:
            heads = range(4) if latent else range(2)       # the query heads of the kv head
            for h in heads:
                assert not np.isfinite(got[i, h, 3]), (i, h)
    if not latent:
        assert torch.equal(out[6], want[6]) and torch.equal(out[8], want[8]) and torch.isnan(out[7, :2]).all()
        assert torch.equal(out[7, 2:], want[7, 2:])


def test_extreme_logits():
    """Rows whose logits rise by far along the context, and logits of thousands: nothing overflows."""
    def edit(ks, vs, q):
        ks[0] *= np.linspace(0.01, 40, ks[0].shape[0])[:, None, None]
        ks[0][:] = bf16(ks[0])
    run_and_check(Paged(13, [1500], [3], 4, 1, 128, 64, edit=edit))

    def falling(ks, vs, q):
        ks[0] *= np.linspace(40, 0.01, ks[0].shape[0])[:, None, None]
        ks[0][:] = bf16(ks[0])
        vs[0][:] = ks[0][..., :512]
    run_and_check(Paged(14, [1500], [3], 4, latent=512, edit=falling))


def test_more_work_than_a_batch_can_have():
    """cu_seqlens that falls and rises again: 300 requests of all 4096 tokens, more units than 31 bits hold.  Nothing is done."""
    T, B, slots, P = 4096, 600, 131072, 64
    p = C.make_attn_params(num_reqs=B, num_q_heads=32, num_kv_heads=8, head_dim=64, page_size=P, total_tokens=T, max_seqlen=slots,
                           num_pages=1, max_pages_per_req=slots // P, max_new_tokens=1)
    q = torch.zeros(T, 32, 64, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(1, P, 8, 64, dtype=torch.bfloat16, device=DEV)
    out, st = torch.full_like(q, 3.0), new_status()
    tables = torch.full((B, slots // P), -1, dtype=torch.int32, device=DEV)
    C.cosa_tree_attention(p, q, i32([0] + [T, 0] * (B // 2)), cache, cache, tables, i32([slots] * B), out=out, status=st)
    torch.cuda.synchronize()
    assert int(st) == -6 and (out == 3.0).all()


# ---- more than 32 query rows to a kv head, which lie a row to a lane
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new", [([40, 7, 300], [40, 7, 33]), ([700, 64, 130], [64, 64, 1]), ([20011, 90, 70], [64, 17, 3])])
def test_many_rows(lens, new, d):
    run_and_check(Paged(31, lens, new, 8, 2, d, 16, tree=True))
    run_and_check(Paged(32, lens, new, 8, 2, d, 32, tree=True, ragged=True, missing=[(0, 0), (1, 1), (2, 2)]))
    run_and_check(Paged(33, lens, new, 14, 2, d, 128, strided="heads"))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("ctx", [100, 9000])
def test_many_rows_and_what_they_do_not_see(d, bad, ctx):
    """The values of new token 5 are not finite, nor are the keys of token 9."""
    n = 20

    def edit(ks, vs, q):
        vs[0][ctx + 5, 0, 3] = vs[0][ctx + 5, 0, d - 1] = bad
        ks[0][ctx + 9, 1] = np.nan
    c, clean = (Paged(34, [ctx + n], [n], 8, 2, d, 64, tree=True, edit=e) for e in (edit, None))
    assert c.masks == clean.masks
    out, lse = c.buffers()
    want, want_lse = clean.buffers()
    c.call(out=out, lse=lse)
    clean.call(out=want, lse=want_lse)
    got = to_f64(out)
    for i, m in enumerate(c.masks[0]):
        if m >> 5 & 1:
            assert not np.isfinite(got[i, :4, [3, d - 1]]).any()
            keep = [e for e in range(d) if e not in (3, d - 1)]
            assert torch.equal(out[i, :4][:, keep], want[i, :4][:, keep]) and torch.equal(lse[i, :4], want_lse[i, :4])
        else:
            assert torch.equal(out[i, :4], want[i, :4]) and torch.equal(lse[i, :4], want_lse[i, :4])
        if m >> 9 & 1:
            assert np.isnan(got[i, 4:]).all()
        else:
            assert torch.equal(out[i, 4:], want[i, 4:]) and torch.equal(lse[i, 4:], want_lse[i, 4:])


def test_many_rows_of_rising_logits():
    """References that move many times, in one CTA and in several."""
    def edit(ks, vs, q):
        ks[0] *= np.linspace(0.01, 40, ks[0].shape[0])[:, None, None]
        ks[0][:] = bf16(ks[0])
    for lens in ([1500], [12000]):
        run_and_check(Paged(35, lens, [20], 4, 1, 128, 64, edit=edit, tree=True))


@pytest.mark.parametrize("group", [4, 1])
def test_bits_behind_the_last_token_count_for_nothing(group):
    """Masks with every bit set: a row sees its request's tokens and no slot behind them."""
    c = Paged(36, [70, 200], [20, 9], 2 * group, 2, 64, 64, tree=True)
    c.masks = [[(1 << n) - 1] * n for n in c.new]
    c.mask = torch.full_like(c.mask, -1)
    run_and_check(c)


@pytest.mark.parametrize("latent", [0, 512])
def test_contradictions(latent):
    """A request whose lengths contradict each other has no keys; the others are as ever."""
    def fresh():
        return Paged(15, [100, 50, 200], [3, 4, 2], 4, 2 if not latent else 1, 64, 16, latent=latent, tree=True)
    for bad in (3, -1, 10 ** 6):
        c = fresh()
        c.kv_len = i32([100, bad, 200])
        out, lse = c.buffers()
        st = new_status()
        c.call(out=out, lse=lse, status=st)
        torch.cuda.synchronize()
        assert int(st) == -6
        assert not out[3:7].any() and torch.isneginf(lse[3:7]).all()
        c.check(out, lse, skip=(1,))
    # a tree too wide
    c = Paged(16, [100, 300], [3, 70], 4, 2 if not latent else 1, 64, 16, latent=latent)
    c.mask = torch.full((76,), -1, dtype=torch.int64, device=DEV)
    c.masks = [[7] * 3, None]
    out, lse = c.buffers()
    st = new_status()
    c.call(out=out, lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st) == -6 and not out[3:73].any() and torch.isneginf(lse[3:73]).all()
    c.check(out, lse, skip=(1,))
    # rows that the tensors do not have are not written
    c = fresh()
    c.cu = i32([0, 3, 7, 4000])
    out, lse = c.buffers()
    guard, st = out.clone(), new_status()
    c.call(out=out, lse=lse, status=st)
    torch.cuda.synchronize()
    assert int(st) == -6 and torch.equal(out[7:], guard[7:])
    c.check(out[:7], lse[:7], skip=(2,))


@pytest.mark.parametrize("latent", [0, 512])
def test_same_bits_every_run(latent):
    c = Paged(17, [3000, 150, 800], [5, 2, 7], 8, 2 if not latent else 1, 128, 64, latent=latent, tree=True)
    first, first_lse = run_and_check(c)
    for _ in range(5):
        ws = torch.randint(0, 256, (max(C.cosa_tree_attention_workspace_size(c.p), C.cosa_latent_attention_workspace_size(c.p)),),
                           dtype=torch.uint8, device=DEV)
        out, lse = run_and_check(c, workspace=ws)
        assert torch.equal(out[:c.T], first[:c.T]) and torch.equal(lse[:c.T], first_lse[:c.T])


# ---------------------------------------------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("row,P,two", [(1024, 64, True), (576, 16, False), (64, 128, True), (8, 32, False), (2056, 16, True)])
def test_commit(row, P, two):
    rng = np.random.default_rng(row + P)
    lens, new = [100, 64, 5, 300, 70, 40], [20, 64, 0, 33, 1, 40]
    paths = [sorted(rng.choice(n, size=int(rng.integers(0, n + 1)), replace=False).tolist()) if n else [] for n in new]
    paths[1], paths[4], paths[5] = list(range(64)), [0], list(range(1, 40))
    pages = max(-(-n // P) for n in lens)
    total = len(lens) * pages + 2
    t = table(rng, len(lens), pages, total, [(3, (300 - 33) // P)] if P < 128 else [])
    caches = [bf(rng, total, P, row) for _ in range(2 if two else 1)]
    before = [to_f64(x) for x in caches]
    path = np.full((len(lens), 64), -7)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    p = C.make_attn_params(num_reqs=len(lens), num_q_heads=1, page_size=P, max_seqlen=pages * P, num_pages=total, max_pages_per_req=pages,
                           max_new_tokens=64)
    st = new_status()
    got = C.cosa_tree_commit(p, caches, cu_of(new), i32(t), i32(lens), i32(path), i32([len(x) for x in paths]), status=st)
    ok(st)
    assert got.tolist() == [n - m + len(x) for n, m, x in zip(lens, new, paths)]
    for x, old in zip(caches, before):
        want = old.copy()
        for b, n in enumerate(lens):
            slots = np.arange(n)
            there = there_of(t, b, n, P, total)
            phys = np.where(there, t[b][slots // P], 0)
            rows = ref.commit(old[phys, slots % P], there, n, new[b], paths[b])
            want[phys[there], (slots % P)[there]] = rows[there]
        assert np.array_equal(to_f64(x), want)


def test_commit_contradictions():
    rng = np.random.default_rng(4)
    lens = [50] * 8
    new = [10] * 8
    t = table(rng, 8, 4, 32)
    path = [[0, 2, 4], [0, 2, 2], [3, 2, 9], [0, 5, 10], [-1, 0, 1], [1, 3, 9], [0, 1, 2], [1, 2, 3]]
    m = [3, 3, 3, 3, 3, -1, 3, 4]
    kv = [50, 50, 50, 50, 50, 50, 9, 50]
    cache = bf(rng, 32, 16, 64)
    before = cache.clone()
    p = C.make_attn_params(num_reqs=8, num_q_heads=1, page_size=16, max_seqlen=64, num_pages=32, max_pages_per_req=4, max_new_tokens=3)
    st = new_status()
    got = C.cosa_tree_commit(p, [cache], cu_of(new), i32(t), i32(kv), i32(path), i32(m), status=st)
    torch.cuda.synchronize()
    assert int(st) == -6 and got.tolist() == [43, 50, 50, 50, 50, 50, 9, 50]
    changed = (cache != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {int(x) for x in t[0]} and changed


# ---------------------------------------------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("H,latent,P,inter,weighted,rows,paged,with_q", [
    (32, 512, 64, False, True, True, True, True), (16, 512, 16, True, True, False, True, True), (5, 256, 128, True, False, True, False, True),
    (1, 256, 32, False, True, False, True, True), (128, 512, 64, True, True, True, True, True), (33, 256, 16, False, True, True, True, True),
    (3, 512, 64, False, True, True, True, False)])
def test_latent_rope(H, latent, P, inter, weighted, rows, paged, with_q):
    rng = np.random.default_rng(H + latent + P)
    lens, starts, spare = [1, 0, 17, 2 * P + 3, 0, 5], [3, 9, P - 2, 0, 0, 4 * P], 3
    T = sum(lens)
    pages = max(-(-(s + n) // P) for s, n in zip(starts, lens))
    total = len(lens) * pages + 2
    t = table(rng, len(lens), pages, total, [(3, 1), (2, 1)])
    wide = bf(rng, T + spare, latent + 64 + 24)
    kv = wide[:, 8:8 + latent + 64]
    q = bf(rng, T + spare, H, 128 + 64)[..., 128:] if with_q else None
    w = bf(rng, latent) * 0.2 + 1 if weighted else None
    inv = torch.from_numpy(1e6 ** (-np.arange(32) / 32)).to(DEV)
    p = C.make_attn_params(num_reqs=len(lens), num_q_heads=H, latent_dim=latent, page_size=P, total_tokens=T + spare, max_seqlen=pages * P,
                           num_pages=total, max_pages_per_req=pages, interleaved=inter)
    cache = garbage(rng, *C.latent_cache_shape(total, P, latent)) if paged else None
    before = None if cache is None else cache.clone()
    q_out = bf(rng, T + spare, H, 64) if with_q else None
    c_out, k_out = (bf(rng, T + spare, latent), bf(rng, T + spare, 64)) if rows else (None, None)
    guards = [None if x is None else x.clone() for x in (q_out, c_out, k_out)]
    st = new_status()
    got = C.cosa_latent_rope(p, kv, cu_of(lens), inv, q=q, weight=w, start=i32(starts), q_out=q_out, c_out=c_out, k_out=k_out, cache=cache,
                             page_table=i32(t) if paged else None, status=st)
    ok(st)
    assert all(a is b for a, b in zip(got, (q_out, c_out, k_out)))
    pos = np.concatenate([np.arange(n) + s for s, n in zip(starts, lens)])
    x = to_f64(kv)[:T]
    cn = ref.norm(x[:, :latent], None if w is None else to_f64(w), 1e-6)
    kr, kmag = ref.rotate(x[:, None, latent:], pos, inv.cpu().numpy(), inter)

    def close(a, b, mag):        # half a bf16 step, and what tests/test_gpu_kv.py derives for norms and rotations
        assert (np.abs(a - b) <= np.abs(b) * 2.0 ** -8 + mag * 2.0 ** -16).all(), float(np.abs(a - b).max())

    if with_q:
        want, mag = ref.rotate(to_f64(q)[:T], pos, inv.cpu().numpy(), inter)
        close(to_f64(q_out)[:T], want, mag)
    if rows:
        close(to_f64(c_out)[:T], cn, np.abs(cn))
        close(to_f64(k_out)[:T], kr[:, 0], kmag[:, 0])
    for x, g in zip((q_out, c_out, k_out), guards):
        assert x is None or torch.equal(x[T:], g[T:])
    if not paged:
        return
    host, row = to_f64(cache), 0
    untouched = torch.ones(total, P, dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(n):
            s = starts[b] + i
            phys = int(t[b, s // P])
            if 0 <= phys < total:
                close(host[phys, s % P, :latent], cn[row + i], np.abs(cn[row + i]))
                close(host[phys, s % P, latent:], kr[row + i, 0], kmag[row + i, 0])
                untouched[phys, s % P] = False
        row += n
    assert torch.equal(cache[untouched].view(torch.int16), before[untouched].view(torch.int16))


@pytest.mark.parametrize("T", [1, 2, 5, 64, 1300, 20000])
def test_latent_rope_sizes_and_far_positions(T):
    rng = np.random.default_rng(T)
    kv, q = bf(rng, T, 576), bf(rng, T, 20, 64)
    inv = torch.from_numpy(1e4 ** (-np.arange(32) / 32)).to(DEV)
    inv[3], inv[7] = 5000.0, 1e-12            # unusual frequencies
    pos = rng.integers(0, 10 ** 6, T)
    p = C.make_attn_params(num_reqs=1, num_q_heads=20, total_tokens=T)
    mine = q.clone()
    got_q, c, k = C.cosa_latent_rope(p, kv, i32([0, T]), inv, q=mine, positions=i32(pos), q_out=mine)
    want, mag = ref.rotate(to_f64(q), pos, inv.cpu().numpy(), False)
    # a turn of 5000 rad times 10^6 is known to 2^-52 of it in the reference's doubles: 2^-19 rad
    assert (np.abs(to_f64(got_q) - want) <= np.abs(want) * 2.0 ** -8 + mag * 2.0 ** -16).all()
    want, mag = ref.rotate(to_f64(kv)[:, None, 512:], pos, inv.cpu().numpy(), False)
    assert (np.abs(to_f64(k) - want[:, 0]) <= np.abs(want[:, 0]) * 2.0 ** -8 + mag[:, 0] * 2.0 ** -16).all()
    assert torch.equal(c, kv[:, :512])        # no weight: as it was


def test_latent_rope_leaves_out_what_does_not_fit():
    rng = np.random.default_rng(2)
    kv, q = bf(rng, 10, 576), bf(rng, 10, 4, 64)
    inv = torch.from_numpy(1e4 ** (-np.arange(32) / 32)).to(DEV)
    p = C.make_attn_params(num_reqs=2, num_q_heads=4, total_tokens=10, page_size=16, max_seqlen=32, num_pages=4, max_pages_per_req=2)
    cache = bf(rng, 4, 16, 576)
    before, q_out, st = cache.clone(), bf(rng, 10, 4, 64), new_status()
    guard = q_out.clone()
    C.cosa_latent_rope(p, kv, i32([0, 4, 8]), inv, q=q, q_out=q_out, start=i32([-2, 30]), cache=cache, page_table=i32([[0, 1], [2, 3]]), status=st)
    torch.cuda.synchronize()
    assert int(st) == -6
    wrote = [i for i in range(10) if not torch.equal(q_out[i], guard[i])]
    assert wrote == [2, 3, 4, 5]
    rows = (cache != before).any(-1).nonzero().tolist()
    assert rows == [[0, 0], [0, 1], [3, 14], [3, 15]]


# ---------------------------------------------------------------------------------------------------------------
# the expanded form
# ---------------------------------------------------------------------------------------------------------------
def expand_case(seed, lens, ctx, H, d, fused=True, spare=2, scale=None, edit=None):
    rng = np.random.default_rng(seed)
    T, totals = sum(lens), [n + c for n, c in zip(lens, ctx)]
    Tk = sum(totals)
    q = bf(rng, T + spare, H, d + 64)
    kv = bf(rng, Tk + spare, H, 2 * d)
    kr = bf(rng, Tk + spare, 64)
    if edit is not None:
        edit(q, kv, kr)
    qn, qr, kn, v = q[..., :d], q[..., d:], kv[..., :d], kv[..., d:]
    if not fused:
        qn, qr, kn, v = (x.contiguous() for x in (qn, qr, kn, v))
    p = C.make_attn_params(num_reqs=len(lens), num_q_heads=H, head_dim=d, total_tokens=T + spare, total_kv_tokens=Tk + spare,
                           max_new_tokens=max(1, max(lens)), sm_scale=scale or (d + 64) ** -0.5)
    return dict(p=p, args=(qn, qr, kn, kr, v, cu_of(lens)), cu_kv=cu_of(totals), lens=lens, totals=totals, rng=rng, T=T, spare=spare, H=H, d=d)


def expand_check(c, out, lse, skip=()):
    qn, qr, kn, kr, v, _ = (to_f64(x) for x in c["args"])
    q = np.concatenate([qn, qr], -1)
    k = np.concatenate([kn, np.broadcast_to(kr[:, None], (*kn.shape[:2], 64))], -1)
    out, lse = to_f64(out), to_f64(lse)
    row = at = 0
    for b, (n, m) in enumerate(zip(c["lens"], c["totals"])):
        if b not in skip:
            seen = np.tril(np.ones((n, m), bool), m - n)
            near(out[row:row + n], lse[row:row + n], *ref.attention(q[row:row + n], k[at:at + m], v[at:at + m], seen, c["p"].sm_scale), m)
        row, at = row + n, at + m


def expand_run(c, check=True, **kw):
    out, lse = bf(c["rng"], c["T"] + c["spare"], c["H"], c["d"]), torch.randn(c["T"] + c["spare"], c["H"], device=DEV)
    guard, guard_lse, st = out.clone(), lse.clone(), new_status()
    kw.setdefault("cu_kv", c["cu_kv"])
    got = C.cosa_latent_prefill(c["p"], *c["args"], out=out, lse=lse, status=st, **kw)
    ok(st)
    assert got is out
    if check:
        expand_check(c, out, lse)
    assert torch.equal(out[c["T"]:], guard[c["T"]:]) and torch.equal(lse[c["T"]:], guard_lse[c["T"]:])
    return out, lse


@pytest.mark.parametrize("H,d,fused", [(4, 128, True), (3, 64, True), (1, 128, False), (16, 64, False)])
def test_prefill(H, d, fused):
    expand_run(expand_case(H + d, [1, 0, 129, 256, 17, 300], [0, 5, 0, 0, 200, 33], H, d, fused))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 257, 513])
def test_prefill_lengths(n, d):
    expand_run(expand_case(n, [n], [0], 2, d))
    expand_run(expand_case(n, [n], [131], 2, d))


@pytest.mark.parametrize("H", [1, 15, 17, 33])
def test_prefill_of_many_heads_and_requests(H):
    """Groups of heads with fewer in the last; requests of every length, more of them than a warp has lanes and fewer."""
    expand_run(expand_case(H, [130, 300, 1, 257], [700, 0, 400, 129], H, 64))
    if H < 16:
        rng = np.random.default_rng(H)
        for B in (31, 32, 33, 70):
            lens = [int(x) for x in rng.integers(0, 290, B)]
            expand_run(expand_case(B, lens, [int(x) for x in rng.integers(0, 200, B)], 2, 64))


def test_prefill_head_by_head():
    """Keys and values as batched products leave them: tokens within a head."""
    c = expand_case(4, [40, 200], [0, 9], 3, 128)
    c["args"] = (*(x.transpose(0, 1).contiguous().transpose(0, 1) for x in c["args"][:3]), c["args"][3],
                 c["args"][4].transpose(0, 1).contiguous().transpose(0, 1), c["args"][5])
    expand_run(c)


def test_prefill_without_cu_kv():
    c = expand_case(5, [40, 200], [0, 0], 2, 128)
    a, _ = expand_run(c)
    b, _ = expand_run(c, cu_kv=None)
    assert torch.equal(a[:240], b[:240])


def test_prefill_logits_that_rise_and_fall():
    for ramp in (torch.linspace(0.01, 40, 902), torch.linspace(40, 0.01, 902)):
        def edit(q, kv, kr):
            kv[..., :128] *= ramp.to(DEV, torch.bfloat16)[:, None, None]
        expand_run(expand_case(6, [900], [0], 1, 128, edit=edit))


def test_prefill_future_is_not_seen():
    """Keys and values of later tokens, of the next request and behind the last that are not finite change nothing."""
    c = expand_case(7, [140, 100], [0, 30], 2, 128)
    want, want_lse = expand_run(c)
    qn, qr, kn, kr, v, _ = c["args"]
    for x in (kn, kr, v):
        x[100:140] = float("nan")
        x[140 + 30 + 60:140 + 130] = float("inf")
        x[270:] = float("nan")
    out, lse = expand_run(c, check=False)
    assert torch.equal(out[:100], want[:100]) and torch.equal(lse[:100], want_lse[:100])
    assert torch.equal(out[140:200], want[140:200]) and torch.equal(lse[140:200], want_lse[140:200])
    assert torch.isnan(out[101:140]).all()


def test_prefill_contradictions():
    c = expand_case(8, [50, 60, 70], [0, 10, 0], 2, 64)
    for cu_kv in ([0, 50, 100, 170], [0, 50, 120, 500]):
        out, lse = bf(c["rng"], 182, 2, 64), torch.randn(182, 2, device=DEV)
        st = new_status()
        C.cosa_latent_prefill(c["p"], *c["args"], cu_kv=i32(cu_kv), out=out, lse=lse, status=st)
        torch.cuda.synchronize()
        assert int(st) == -6
        bad = slice(50, 110) if cu_kv[2] == 100 else slice(110, 180)
        assert not out[bad].any() and torch.isneginf(lse[bad]).all()
        if cu_kv[2] == 120:
            expand_check(c, out, lse, skip=(2,))


def test_prefill_same_bits_every_run():
    c = expand_case(9, [700, 300], [0, 100], 4, 128)
    a, la = expand_run(c)
    for _ in range(4):
        b, lb = expand_run(c)
        assert torch.equal(a[:1000], b[:1000]) and torch.equal(la[:1000], lb[:1000])
