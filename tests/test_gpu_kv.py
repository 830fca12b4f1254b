"""The calls of include/cosa_kv.h on the GPU against tests/kv_reference.py.

Tolerances.  A bf16 output is off by half a step at most, 2^-8 of its value.  On top:
  norm and rotation   the mean square sums at most 128 squares in fp32 (2^-17 of it at worst), its root halves that; the
                      angle's turns are reduced in 64 bits and rounded to fp32 (below 2^-23), sine and cosine are good to
                      a few 2^-24: 2^-16 of |a| + |b| covers all of it.
  attention           p * s is rounded to bf16, 2^-8 of each term: 2^-8 of sum p |v|; a logit off by e changes p by at most
                      a factor exp(2 e) (numerator and sum): 2.1 e of sum p |v| for the e of kv_reference.logit_error;
                      the fp32 sums lose 48 2^-24 of sum p |v|, in that 2^-8's shadow: 2^-17 of it.
  weights             a sum of fp32 products: 2.1 e + 2^-18 of the added part (ex2.approx is good to 2^-22, the argument
                      of at most 2^7 to 2^-17 * ln 2 / 2), and 2^-23 of the total.
4-bit values, kept slots and moved rows are exact.
"""
import numpy as np
import pytest
import torch

from block_sparse_long_gb300 import cosa, kv as C
from tests import kv_reference as ref
from tests.kv_helpers import bf, cu_of, exists, i32, new_status, noise_cache, ok, packed, table

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_long_gb300 import build
    build.build()


def near(got, want, slack):
    """|got - want| <= half a bf16 step of want + slack, and the same NaN and infinities."""
    got = ref.to_f64(got) if isinstance(got, torch.Tensor) else got
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    slack = np.broadcast_to(np.asarray(slack, dtype=np.float64), want.shape)
    off = np.abs(got - want)[fine] - np.abs(want)[fine] * 2.0 ** -8 - slack[fine]
    assert not off.size or off.max() <= 1e-30, float(off.max())


# ---------------------------------------------------------------------------------------------------------------
# norm, rotation, bf16 cache write
# ---------------------------------------------------------------------------------------------------------------
def rope_case(seed, lens, starts, Hq, Hkv, d, P, rot, inter, norm=True, spare_rows=3, missing=(), fused=True, far=0, eps=1e-6):
    rng = np.random.default_rng(seed)
    T = sum(lens)
    if fused:
        qkv = bf(rng, T + spare_rows, (Hq + 2 * Hkv) * d)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    else:
        q, k, v = bf(rng, T + spare_rows, Hq, d), bf(rng, T + spare_rows, Hkv, d), bf(rng, T + spare_rows, Hkv, d)
    wq, wk = ((bf(rng, d) * 0.2 + 1) if norm else None for _ in range(2))
    inv = torch.from_numpy(1e6 ** (-np.arange(rot // 2) / (rot // 2))).to(DEV)
    pages = max(1, max(-(-(s + n) // P) for s, n in zip(starts, lens)))
    t = table(rng, len(lens), pages, len(lens) * pages + 2, missing)
    pos = np.concatenate([np.arange(n) + s + far for s, n in zip(starts, lens)] + [np.full(spare_rows, 7)])
    p = C.make_kv_params(num_reqs=len(lens), num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, page_size=P, total_tokens=T + spare_rows,
                         max_seqlen=pages * P, num_pages=len(lens) * pages + 2, max_pages_per_req=pages, rotary_dim=rot,
                         interleaved=inter, norm_eps=eps)
    return dict(p=p, q=q, k=k, v=v, wq=wq, wk=wk, inv=inv, t=t, pos=pos, lens=lens, starts=starts, T=T, P=P, d=d,
                norm=norm, inter=inter, rng=rng, eps=eps)


def rope_want(c):
    w = [None if x is None else ref.to_f64(x) for x in (c["wq"], c["wk"])]
    inv = c["inv"].cpu().numpy()
    return [ref.norm_rope(ref.to_f64(x)[:c["T"]], w[i], c["pos"][:c["T"]], inv, c["inter"], c["eps"]) for i, x in enumerate((c["q"], c["k"]))]


@pytest.mark.parametrize("Hq,Hkv,d,P,rot,inter,norm", [
    (32, 8, 128, 64, 128, False, True), (4, 4, 64, 16, 64, False, True), (7, 1, 128, 128, 64, False, False),
    (12, 4, 64, 32, 16, True, True), (3, 3, 128, 16, 128, True, False), (5, 1, 64, 64, 48, False, True),
    (6, 2, 128, 32, 112, True, True)])
def test_rope_to_pages(Hq, Hkv, d, P, rot, inter, norm):
    lens, starts = [1, 0, 17, 2 * P + 3, 0, 5], [3, 9, P - 2, 0, 0, 4 * P]
    c = rope_case(Hq * 100 + d + rot, lens, starts, Hq, Hkv, d, P, rot, inter, norm, missing=[(3, 1), (2, 1)])
    total = c["p"].num_pages
    kc, vc = bf(c["rng"], total, P, Hkv, d), bf(c["rng"], total, P, Hkv, d)
    before = kc.clone(), vc.clone()
    q_out = bf(c["rng"], c["p"].total_tokens, Hq, d)
    guard = q_out.clone()
    st = new_status()
    got, none = C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], cu_of(lens), c["inv"], v=c["v"], q_weight=c["wq"], k_weight=c["wk"],
                                    positions=i32(c["pos"]), start=i32(starts), q_out=q_out, k_cache=kc, v_cache=vc,
                                    page_table=i32(c["t"]), status=st)
    ok(st)
    assert got is q_out and none is None
    (yq, mq), (yk, mk) = rope_want(c)
    near(got[:c["T"]], yq, mq * 2.0 ** -16)
    assert torch.equal(got[c["T"]:], guard[c["T"]:])                 # rows behind the last request
    row = 0
    want_v = before[1].clone()
    untouched = torch.ones(total, P, dtype=torch.bool)
    k_np = ref.to_f64(kc)
    for b, n in enumerate(lens):
        for i in range(n):
            s = starts[b] + i
            phys = int(c["t"][b, s // P])
            if 0 <= phys < total:
                near(k_np[phys, s % P], yk[row + i], mk[row + i] * 2.0 ** -16)
                want_v[phys, s % P] = c["v"][row + i]
                untouched[phys, s % P] = False
        row += n
    assert torch.equal(vc, want_v)
    assert torch.equal(kc[untouched], before[0][untouched])


@pytest.mark.parametrize("T", [1, 2, 5, 64, 1300])
def test_rope_to_rows_far_positions(T):
    """Decode rows; positions up to 10^6 rad and more: the angles keep their accuracy."""
    lens = [1] * T if T < 100 else [T]
    c = rope_case(T, lens, [0] * len(lens), 8, 2, 128, 16, 128, False, spare_rows=0, far=1_048_000)
    st = new_status()
    q_out, k_out = C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], cu_of(lens), c["inv"], q_weight=c["wq"], k_weight=c["wk"],
                                       positions=i32(c["pos"]), status=st)
    ok(st)
    for got, (y, m) in zip((q_out, k_out), rope_want(c)):
        near(got, y, m * 2.0 ** -16)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_any_frequency(inter):
    """Zero, negative, far larger and far smaller frequencies than usual, at both sides of where their arithmetic changes, and
    negative positions; what is not finite gives NaN.  (Up to 2^53 the double of position * frequency in the reference is
    exact to half a step: the positions here leave it 2^-20 of a radian at worst, in the 2^-16's shadow.)"""
    c = rope_case(31, [900], [0], 4, 2, 128, 16, 128, inter, spare_rows=0)
    rng = np.random.default_rng(32)
    inv = np.concatenate([[0.0, -0.0, 1.0, -1.0, 0.5, 2.0 ** -36, -2.0 ** -37, 2.0 ** -60, 5e-324, 1024.0, 1023.9999, -1024.5, 5000.0],
                          (2.0 ** rng.uniform(-40, 11, 51)) * rng.choice([-1, 1], 51)])
    c["inv"] = torch.from_numpy(inv).to(DEV)
    c["pos"] = np.concatenate([[0, 1, -1, 2 ** 20, -2 ** 20], rng.integers(-2 ** 20, 2 ** 20, 895)])
    for scale in (1, 2 ** 10):                                      # with small frequencies, the farthest positions
        if scale > 1:
            c["inv"], c["pos"] = c["inv"] / 2 ** 14, np.clip(c["pos"] * 2 ** 11, -2 ** 31, 2 ** 31 - 1)
        st = new_status()
        got = C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], cu_of([900]), c["inv"], q_weight=c["wq"], k_weight=c["wk"],
                                  positions=i32(c["pos"]), status=st)
        ok(st)
        for x, (y, m) in zip(got, rope_want(c)):
            near(x, y, m * 2.0 ** -16)
    c["inv"][[0, 5, 9]] = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=torch.float64, device=DEV)
    got = C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], cu_of([900]), c["inv"], q_weight=c["wq"], k_weight=c["wk"],
                              positions=i32(c["pos"]))[0]
    bad = [2 * f + e for f in (0, 5, 9) for e in (0, 1)] if inter else [f + e for f in (0, 5, 9) for e in (0, 64)]
    assert (torch.isnan(got).sum((0, 1)) == 0).nonzero().flatten().tolist() == [i for i in range(128) if i not in bad]
    assert torch.isnan(got[..., bad]).all()


@pytest.mark.parametrize("Hq,Hkv,d,rot,T,inter,paged", [(3, 1, 64, 64, 20001, False, False), (2, 1, 64, 32, 20003, True, True),
                                                        (5, 1, 64, 64, 12345, False, True), (2, 2, 128, 128, 9999, False, False),
                                                        (3, 1, 128, 48, 9731, True, True), (6, 2, 128, 128, 8001, False, True),
                                                        (13, 1, 64, 48, 8003, True, False)])
def test_rope_several_tokens_per_warp(Hq, Hkv, d, rot, T, inter, paged):
    """Many tokens, the first five with so few heads that a warp has several: they lie in different requests, empty ones
    between them, and the last warp has fewer."""
    lens = [1, 0, 0, 2, 1, 1, 0, 5, 3, 1, 1, 1, 0, T - 16]
    starts = [(5 * b) % 13 for b in range(len(lens))]
    c = rope_case(T, lens, starts, Hq, Hkv, d, 128, rot, inter, spare_rows=2)
    st = new_status()
    args = dict(q_weight=c["wq"], k_weight=c["wk"], positions=i32(c["pos"]), start=i32(starts), status=st)
    (yq, mq), (yk, mk) = rope_want(c)
    if not paged:
        q_out, k_out = C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], cu_of(lens), c["inv"], **args)
        ok(st)
        near(k_out[:c["T"]], yk, mk * 2.0 ** -16)
    else:
        kc = torch.zeros(c["p"].num_pages, 128, Hkv, d, dtype=torch.bfloat16, device=DEV)
        vc = torch.zeros_like(kc)
        q_out, _ = C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], cu_of(lens), c["inv"], v=c["v"], k_cache=kc, v_cache=vc,
                                       page_table=i32(c["t"]), **args)
        ok(st)
        slots = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, lens)])
        reqs = np.repeat(np.arange(len(lens)), lens)
        at = c["t"][reqs, slots // 128].astype(np.int64) * 128 + slots % 128
        near(ref.to_f64(kc).reshape(-1, Hkv, d)[at], yk, mk * 2.0 ** -16)
        assert torch.equal(vc.flatten(0, 1)[torch.from_numpy(at).to(DEV)], c["v"][:c["T"]])
        rest = np.ones(c["p"].num_pages * 128, bool)
        rest[at] = False
        assert not bool(kc.flatten(0, 1)[torch.from_numpy(rest).to(DEV)].any())
    near(q_out[:c["T"]], yq, mq * 2.0 ** -16)


def test_rope_positions_default_to_slots_and_both_outputs():
    lens, starts = [4, 9], [30, 2]
    c = rope_case(5, lens, starts, 4, 2, 64, 16, 32, False, spare_rows=0)
    kc, vc = (torch.zeros(c["p"].num_pages, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k_out = torch.zeros(13, 2, 64, dtype=torch.bfloat16, device=DEV)
    st = new_status()
    q_out, ko = C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], cu_of(lens), c["inv"], v=c["v"], q_weight=c["wq"], k_weight=c["wk"],
                                    start=i32(starts), k_out=k_out, k_cache=kc, v_cache=vc, page_table=i32(c["t"]), status=st)
    ok(st)
    assert ko is k_out
    (yq, mq), (yk, mk) = rope_want(c)
    near(q_out, yq, mq * 2.0 ** -16)
    near(k_out, yk, mk * 2.0 ** -16)
    row = 0
    for b, n in enumerate(lens):
        for i in range(n):
            s = starts[b] + i
            assert torch.equal(kc[int(c["t"][b, s // 16]), s % 16], k_out[row + i])
        row += n


def test_rope_in_place_and_special_values():
    """q_out may be q.  Zero rows stay zero (eps), infinities and NaN stay in their row."""
    c = rope_case(6, [6], [0], 4, 2, 128, 16, 128, False, fused=False, spare_rows=0)
    c["q"][1] = 0
    c["q"][2, 1, 3] = float("nan")
    c["q"][3, 2, 100] = float("inf")
    c["k"][4] *= 1e-30
    c["q"][5, 3] *= 2.0 ** 100                                       # squares overflow fp32: left out below
    y, m = rope_want(c)[0]
    yk, mk = rope_want(c)[1]
    q, k = c["q"].clone(), c["k"].clone()
    C.cosa_qk_norm_rope(c["p"], q, k, cu_of([6]), c["inv"], q_weight=c["wq"], k_weight=c["wk"], positions=i32(c["pos"]),
                        q_out=q, k_out=k)
    got = ref.to_f64(q)
    keep = np.ones((6, 4), bool)
    keep[2, 1] = keep[3, 2] = keep[5, 3] = False
    near(got[keep], y[keep], m[keep] * 2.0 ** -16)
    assert np.isnan(got[2, 1]).all() and np.isnan(got[3, 2, [100, 36]]).all()
    assert (got[5, 3] == 0).all()                                    # 1 / sqrt(inf)
    near(k, yk, mk * 2.0 ** -16)


def test_rope_reports_contradictions():
    c = rope_case(7, [4, 4], [0, 0], 2, 1, 64, 16, 64, False, spare_rows=0)
    kc = torch.zeros(c["p"].num_pages, 16, 1, 64, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    for cu, start in (([0, 4, 9], [0, 0]), ([0, 4, 8], [0, 13]), ([0, 4, 8], [-1, 0])):
        st = new_status()
        kc.zero_()
        C.cosa_qk_norm_rope(c["p"], c["q"], c["k"], i32(cu), c["inv"], v=c["v"], start=i32(start), k_cache=kc, v_cache=vc,
                            page_table=i32(c["t"]), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == cosa.COSA_ERR_BAD_INPUT, (cu, start)


# ---------------------------------------------------------------------------------------------------------------
# 4-bit store and load
# ---------------------------------------------------------------------------------------------------------------
def special(rng, x):
    """Rows that a quantiser can get wrong: zeros, tiny and huge magnitudes, borders, values that are not finite."""
    x[0] = 0
    x[1] *= 2.0 ** -130
    x[2] *= 2.0 ** 120
    x[3] = torch.from_numpy(rng.integers(-14, 15, tuple(x[3].shape)) * 0.5).to(x)       # halves: ties
    x[3, :, 0::32] = 7.0
    x[4, 0, 5] = float("inf")
    x[5, -1, 40] = float("nan")
    x[6, 0, 63] = float("-inf")
    x[7] = torch.from_numpy(2.0 ** rng.integers(-133, -126, tuple(x[7].shape)).astype(np.float64)).to(x)


@pytest.mark.parametrize("H,d,P", [(8, 128, 64), (1, 64, 16), (3, 128, 128), (2, 64, 32), (5, 128, 16)])
def test_store_rows_then_load(H, d, P):
    rng = np.random.default_rng(H * d + P)
    lens, starts = [1, 0, 40, 19, 1, 2 * P], [0, 3, 5, P - 1, 2 * P + 15, P // 2]
    T = sum(lens)
    kv = bf(rng, T + 2, 2 * H * d + 8)
    k, v = kv[:, :H * d].unflatten(1, (H, d)), kv[:, H * d:2 * H * d].unflatten(1, (H, d))
    special(rng, k[4:])
    special(rng, v[20:])
    pages = max(-(-(s + n) // P) for s, n in zip(starts, lens))
    t = table(rng, len(lens), pages, len(lens) * pages + 1, missing=[(2, 0), (5, 1)])
    total = len(lens) * pages + 1
    cache = noise_cache(rng, total, H, P, d)
    want = cache.cpu().numpy().copy()
    p = C.make_kv_params(num_reqs=len(lens), num_q_heads=H, num_kv_heads=H, head_dim=d, page_size=P, total_tokens=T + 2,
                         max_seqlen=pages * P, num_pages=total, num_kv4_pages=total, max_pages_per_req=pages)
    st = new_status()
    C.cosa_kv4_store(p, cache, i32(t), k, v, cu_seqlens=cu_of(lens), start=i32(starts), status=st)
    ok(st)
    kn, vn = ref.to_f64(k), ref.to_f64(v)
    row = 0
    for b, n in enumerate(lens):
        for i in range(n):
            s, phys = starts[b] + i, int(t[b, (starts[b] + i) // P])
            if 0 <= phys < total:
                for h in range(H):
                    ref.pack_slot(want, phys, h, s % P, kn[row + i, h], vn[row + i, h])
        row += n
    # byte for byte, the neighbours' bytes among them
    assert np.array_equal(cache.cpu().numpy(), want)

    # and back: only the slots asked for, through another table
    t16 = table(rng, len(lens), pages, total, missing=[(3, 1)])
    kc, vc = bf(rng, total, P, H, d), bf(rng, total, P, H, d)
    want_k, want_v = ref.to_f64(kc), ref.to_f64(vc)
    ends = [s + n for s, n in zip(starts, lens)]
    C.cosa_kv4_load(p, cache, i32(t), kc, vc, i32(t16), kv_len=i32(ends), start=i32(starts), status=st)
    ok(st)
    for b, (s0, e) in enumerate(zip(starts, ends)):
        for s in range(s0, e):
            a, z = int(t[b, s // P]), int(t16[b, s // P])
            if 0 <= a < total and 0 <= z < total:
                for h in range(H):
                    x, y = ref.unpack_slot(want, a, h, s % P, d)
                    want_k[z, s % P, h], want_v[z, s % P, h] = ref.bf16(x), ref.bf16(y)
    assert np.array_equal(ref.to_f64(kc), want_k, equal_nan=True) and np.array_equal(ref.to_f64(vc), want_v, equal_nan=True)


@pytest.mark.parametrize("H,d,P", [(8, 128, 64), (2, 64, 16), (3, 64, 128)])
def test_store_pages(H, d, P):
    rng = np.random.default_rng(H * d + P + 1)
    ends, starts = [1, 0, 100, 2 * P, 33], [0, 0, 17, P, 40]          # the last one is empty: start behind the end
    pages = max(-(-e // P) for e in ends)
    total = len(ends) * pages + 2
    k, v = bf(rng, total, P, H, d), bf(rng, total, P, H, d)
    special(rng, k[:, 3])
    special(rng, v[:, 5])
    t4, t16 = table(rng, 5, pages, total, missing=[(2, 0)]), table(rng, 5, pages, total, missing=[(3, 1)])
    cache = noise_cache(rng, total, H, P, d)
    want = cache.cpu().numpy().copy()
    p = C.make_kv_params(num_reqs=5, num_q_heads=H, num_kv_heads=H, head_dim=d, page_size=P, max_seqlen=pages * P, num_pages=total,
                         num_kv4_pages=total, max_pages_per_req=pages)
    st = new_status()
    C.cosa_kv4_store(p, cache, i32(t4), k, v, src_page_table=i32(t16), start=i32(starts), kv_len=i32(ends), status=st)
    ok(st)
    kn, vn = ref.to_f64(k), ref.to_f64(v)
    for b, (s0, e) in enumerate(zip(starts, ends)):
        for s in range(s0, e):
            a, z = int(t16[b, s // P]), int(t4[b, s // P])
            if 0 <= a < total and 0 <= z < total:
                for h in range(H):
                    ref.pack_slot(want, z, h, s % P, kn[a, s % P, h], vn[a, s % P, h])
    assert np.array_equal(cache.cpu().numpy(), want)


def test_store_and_load_report_contradictions():
    p = C.make_kv_params(num_reqs=2, num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=16, total_tokens=4, max_seqlen=32,
                         num_pages=4, num_kv4_pages=4, max_pages_per_req=2)
    rng = np.random.default_rng(0)
    cache, t = noise_cache(rng, 4, 1, 16, 64), i32([[0, 1], [2, 3]])
    before = cache.clone()
    k = bf(rng, 4, 1, 64)
    kc = bf(rng, 4, 16, 1, 64)
    for run in (lambda st: C.cosa_kv4_store(p, cache, t, k, k, cu_seqlens=i32([0, 0, 4]), start=i32([0, 30]), status=st),
                lambda st: C.cosa_kv4_store(p, cache, t, k, k, cu_seqlens=i32([0, 0, 5]), start=i32([0, 40]), status=st),
                lambda st: C.cosa_kv4_store(p, cache, t, kc, kc, src_page_table=t, kv_len=i32([0, 33]), status=st),
                lambda st: C.cosa_kv4_store(p, cache, t, kc, kc, src_page_table=t, kv_len=i32([0, -1]), status=st),
                lambda st: C.cosa_kv4_load(p, cache, t, kc, kc.clone(), t, kv_len=i32([0, 5]), start=i32([0, -5]), status=st)):
        st = new_status()
        run(st)
        torch.cuda.synchronize()
        assert int(st.item()) == cosa.COSA_ERR_BAD_INPUT
    # the tokens that fit were stored (30 and 31), nothing else
    changed = (cache != before).flatten(2).any(-1).flatten().tolist()
    assert changed == [False, False, False, True]


# ---------------------------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------------------------
def attend(rng, lens, new, Hq, Hkv, d, P, *, weights=False, missing=(), edit=None, hint=None, scale=None, q_scale=1.5, spare=2, wide=False):
    cache, t, ks, vs = packed(rng, lens, Hkv, P, d, missing=missing, edit=edit)
    if wide:          # a max_seqlen far above the lengths: the batch is shared as one list instead of by clusters
        more = np.full((len(lens), -(-20000 // P)), -1, np.int32)
        more[:, :t.shape[1]] = t
        t = more
    T = sum(new)
    q = bf(rng, T + spare, Hq, d, scale=q_scale)
    pages = t.shape[1]
    p = C.make_kv_params(num_reqs=len(lens), num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, page_size=P, total_tokens=T + spare,
                         max_seqlen=pages * P, num_kv4_pages=cache.shape[0], max_pages_per_req=pages,
                         max_new_tokens=max(1, max(new)) if hint is None else hint, sm_scale=scale)
    acc = torch.from_numpy(rng.random((len(lens), Hkv, pages * P)).astype(np.float32)).to(DEV) if weights else None
    return dict(p=p, q=q, cache=cache, t=t, ks=ks, vs=vs, lens=lens, new=new, acc=acc, T=T, P=P, rng=rng)


def check_attention(c, out, acc, acc0):
    p = c["p"]
    q = ref.to_f64(c["q"])
    row = 0
    g = p.num_q_heads // p.num_kv_heads
    for b, (L, n) in enumerate(zip(c["lens"], c["new"])):
        k, v = c["ks"][b], c["vs"][b]
        there = exists(c["t"], b, L, c["P"], p.num_kv4_pages)
        want, mag, prob = ref.attention(q[row:row + n], k, v, there, p.sm_scale)
        e = ref.logit_error(q[row:row + n], k[there], p.sm_scale)
        near(out[row:row + n], want, mag * (2.0 ** -8 + 2.0 ** -17 + 2.1 * e))
        if acc is not None:
            add = prob.reshape(n, p.num_kv_heads, g, L).sum((0, 2))
            got, was = ref.to_f64(acc[b, :, :L]), ref.to_f64(acc0[b, :, :L])
            assert (np.abs(got - was - add) <= add * (2.1 * e + 2.0 ** -18) + np.abs(was + add) * 2.0 ** -23).all()
            assert torch.equal(acc[b, :, L:], acc0[b, :, L:])
        row += n


def run_attention(c, **kw):
    st = new_status()
    out = bf(c["rng"], *c["q"].shape)
    guard = out.clone()
    acc0 = None if c["acc"] is None else c["acc"].clone()
    got = C.cosa_kv4_attention(c["p"], c["q"], cu_of(c["new"]), c["cache"], i32(c["t"]), i32(c["lens"]), out=out,
                               weights=c["acc"], status=st, **kw)
    ok(st)
    assert got is out and torch.equal(out[c["T"]:], guard[c["T"]:])
    check_attention(c, out, c["acc"], acc0)
    return out


@pytest.mark.parametrize("weights,wide", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("Hq,Hkv,d,P", [(32, 8, 128, 64), (4, 4, 64, 16), (7, 1, 128, 128), (8, 1, 64, 64), (16, 1, 128, 16),
                                        (12, 4, 128, 32), (24, 1, 64, 32), (9, 3, 64, 128), (20, 1, 128, 32), (33, 1, 128, 64)])
def test_attention_lengths(Hq, Hkv, d, P, weights, wide):
    """One token per request; lengths from zero to several tiles; pages that end inside the tile; missing pages."""
    lens = [1, 15, 16, 17, 0, 64, 130, 300, 2, P + 1]
    c = attend(np.random.default_rng(Hq * 7 + d + P), lens, [1] * len(lens), Hq, Hkv, d, P, weights=weights,
               missing=[(7, 0), (6, min(1, 130 // P)), (2, 0)], wide=wide)
    run_attention(c)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,new,hint", [(8, 2, 128, [3, 0, 1, 5, 2], None), (8, 2, 128, [3, 0, 1, 5, 2], 1), (4, 4, 64, [9, 1, 0, 20, 2], None),
                                               (16, 2, 64, [2, 0, 1, 3, 2], 2), (6, 2, 128, [40, 0, 1, 2, 2], 100), (5, 5, 128, [8, 8, 8, 8, 2], 3), (7, 1, 64, [3, 1, 1, 2, 0], None),
                                               (6, 1, 128, [4, 0, 1, 8, 1], None), (12, 1, 128, [2, 2, 2, 2, 2], 1)])
def test_attention_several_tokens(Hq, Hkv, d, new, hint, wide):
    """Causal at the end; more rows than a row tile has; requests without queries; query tokens that see nothing (more
    queries than slots); any hint gives the same."""
    lens = [100, 50, 1, 7, 1]
    c = attend(np.random.default_rng(sum(new) + d), lens, new, Hq, Hkv, d, 16, weights=True, hint=hint, wide=wide)
    run_attention(c)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("L,B,Hkv", [(1000, 1, 8), (5000, 1, 1), (2500, 2, 2), (333, 5, 3)])
def test_attention_split_over_ctas(L, B, Hkv, wide):
    """Long contexts: a (request, kv head) is shared by many CTAs and joined; a run of a CTA spans requests."""
    rng = np.random.default_rng(L)
    run_attention(attend(rng, [L - 37 * b for b in range(B)], [1] * B, 4 * Hkv, Hkv, 64, 64, weights=True, missing=[(0, 2)], wide=wide))


@pytest.mark.parametrize("wide", [False, True])
def test_attention_any_hint(wide):
    """A hint far above the tokens that there are is as good as their number."""
    c = attend(np.random.default_rng(23), [700, 3, 90], [2, 0, 3], 8, 2, 128, 16, weights=True, wide=wide, hint=7)
    acc0, out = c["acc"].clone(), run_attention(c)
    acc1, c["acc"], c["p"].max_new_tokens, c["rng"] = c["acc"], acc0, 2 ** 31 - 1, np.random.default_rng(24)
    assert torch.equal(run_attention(c)[:c["T"]], out[:c["T"]]) and torch.equal(c["acc"], acc1)


def test_attention_large_logits_and_scale():
    """A maximum that moves late by hundreds: the running rescale; one slot takes nearly all of the weight."""
    def edit(b, k, v):
        for s in range(0, len(k), 97):
            k[s] = ref.bf16(k[s] * (1 + s / 100))
    rng = np.random.default_rng(11)
    run_attention(attend(rng, [700, 190], [1, 2], 4, 2, 128, 16, weights=True, edit=edit, scale=0.02, q_scale=4.0))


def test_attention_keeps_nan_where_it_is_seen():
    """A NaN group of a key, of a value: rows that see the slot give NaN (for a value, in its 32 channels); rows that do
    not see it, and slots past the end that hold anything, do not."""
    def edit(b, k, v):
        if b == 0:
            k[10, 0, 3] = np.nan
        if b == 1:
            v[19, 1, 40] = np.inf
    rng = np.random.default_rng(12)
    c = attend(rng, [20, 20, 20], [1, 2, 1], 4, 2, 64, 16, edit=edit)
    out = torch.zeros_like(c["q"])
    C.cosa_kv4_attention(c["p"], c["q"], cu_of(c["new"]), c["cache"], i32(c["t"]), i32(c["lens"]), out=out)
    o = ref.to_f64(out)
    assert np.isnan(o[0, :2]).all() and np.isfinite(o[0, 2:]).all()              # request 0: heads of kv head 0
    assert np.isfinite(o[1]).all()                                               # request 1's first token does not see slot 19
    assert np.isfinite(o[2, :2]).all() and np.isfinite(o[2, 2:, :32]).all() and np.isnan(o[2, 2:, 32:]).all()
    assert np.isfinite(o[3]).all()


def test_attention_reports_contradictions():
    c = attend(np.random.default_rng(13), [30, 30], [1, 1], 2, 1, 64, 16, spare=0)
    good = run_attention(c)
    for cu, lens in (([0, 1, 2], [30, 33]), ([0, 1, 2], [30, -1]), ([0, 1, 3], [30, 30]), ([0, 3, 2], [30, 30])):
        st = new_status()
        out = torch.zeros_like(c["q"])
        C.cosa_kv4_attention(c["p"], c["q"], i32(cu), c["cache"], i32(c["t"]), i32(lens), out=out, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == cosa.COSA_ERR_BAD_INPUT
        if cu == [0, 1, 2]:
            assert torch.equal(out[0], good[0]) and (out[1] == 0).all()          # the other request is served


def test_attention_is_deterministic_and_repeatable():
    c = attend(np.random.default_rng(14), [900, 40, 333], [1, 2, 1], 8, 2, 128, 64, weights=True)
    ws = torch.empty(C.cosa_kv4_attention_workspace_size(c["p"], True), dtype=torch.uint8, device=DEV)
    acc0, outs = c["acc"].clone(), []
    for fill in (0, 255, 7):                                                     # whatever the workspace holds
        ws.fill_(fill)
        acc = acc0.clone()
        out = C.cosa_kv4_attention(c["p"], c["q"], cu_of(c["new"]), c["cache"], i32(c["t"]), i32(c["lens"]), weights=acc, workspace=ws)
        outs.append((out[:c["T"]].clone(), acc))
    for o, a in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(a, outs[0][1])


# ---------------------------------------------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------------------------------------------
def run_evict(rng, lens, H, d, P, budget, sink, recent, *, missing=(), weights=None, st=None):
    pages = max(1, max(-(-n // P) for n in lens))
    room = -(-budget // P)
    B = len(lens)
    t = table(rng, B, pages + room, B * (pages + room) + 2)
    src, dst = t[:, :pages].copy(), t[:, pages:].copy()
    total = B * (pages + room) + 2
    for n, (b, pg) in enumerate(missing):
        src[b, pg] = -1 if n % 2 == 0 else total
    cache = noise_cache(rng, total, H, P, d)
    before = cache.cpu().numpy()
    if weights is None:
        weights = rng.exponential(size=(B, H, pages * P)).astype(np.float32)
    p = C.make_kv_params(num_reqs=B, num_q_heads=H, num_kv_heads=H, head_dim=d, page_size=P, max_seqlen=pages * P, num_kv4_pages=total,
                         max_pages_per_req=pages, budget=budget, sink=sink, recent=recent, max_dst_pages=room)
    status = new_status()
    new_len, kept, w_out = C.cosa_kv4_evict(p, cache, i32(src), i32(lens), torch.from_numpy(weights).to(DEV), i32(dst), status=status)
    ok(status)
    after = cache.cpu().numpy()
    want = before.copy()
    new_len, kept, w_out = new_len.cpu().numpy(), kept.cpu().numpy(), w_out.cpu().numpy()

    def row_bytes(x, phys, h, s):
        """The three pieces of a slot: views into a page's bytes."""
        G = d // 32
        tile = x[phys, h].reshape(-1)[(s % P) // 16 * 18 * d:][:18 * d]
        r = s % 16
        rv = (r % 2) * 8 + r // 2
        return [tile[r * d // 2:(r + 1) * d // 2], tile[8 * d + rv * d // 2:8 * d + (rv + 1) * d // 2],
                tile[16 * d + r * 2 * G:16 * d + (r + 1) * 2 * G], tile[16 * d + 32 * G + r * 2 * G:16 * d + 32 * G + (r + 1) * 2 * G]]

    for b, n in enumerate(lens):
        there = exists(src, b, n, P, total)
        for h in range(H):
            slots = ref.evict(weights[b, h, :n], there, budget, sink, recent)
            assert new_len[b] == len(slots)
            assert np.array_equal(kept[b, h, :len(slots)], slots) and (kept[b, h, len(slots):] == -1).all()
            assert np.array_equal(w_out[b, h, :len(slots)], weights[b, h][slots], equal_nan=True) and (w_out[b, h, len(slots):] == 0).all()
            for j, s in enumerate(slots):
                for a, z in zip(row_bytes(before, int(src[b, s // P]), h, int(s)), row_bytes(want, int(dst[b, j // P]), h, j)):
                    z[:] = a
    assert np.array_equal(after, want)           # sources, neighbours and slots past the kept ones as they were


@pytest.mark.parametrize("H,d,P", [(2, 128, 64), (3, 64, 16), (1, 128, 16), (2, 64, 128)])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 0, 1), (16, 4, 4), (33, 0, 0), (100, 50, 50), (700, 3, 5)])
def test_evict(H, d, P, budget, sink, recent):
    rng = np.random.default_rng(H * d + budget)
    run_evict(rng, [0, 1, 16, 33, 250, 600], H, d, P, budget, sink, recent, missing=[(4, 0), (5, 250 // P), (1, 0)])


def test_evict_ties_signs_and_special_weights():
    rng = np.random.default_rng(20)
    w = rng.integers(-2, 3, (3, 2, 512)).astype(np.float32)          # many ties, zeros of both signs, negatives
    w[0, 0, ::7] = -0.0
    w[1] = 0.5                                                       # all equal
    w[2, 0, ::3] = np.nan
    w[2, 0, 1::3] = np.inf
    w[2, 1, ::2] = -np.inf
    w[2, 1, 1::2] = rng.standard_normal(256) * 1e-42                 # subnormal
    for budget in (5, 100, 300, 511):
        run_evict(rng, [512, 500, 512], 2, 64, 64, budget, 2, 3, weights=w)


@pytest.mark.parametrize("n,budget", [(20000, 3000), (9000, 8999), (5000, 1)])
def test_evict_long(n, budget):
    rng = np.random.default_rng(n)
    run_evict(rng, [n, n // 3], 1, 64, 64, budget, 0, 0)


def test_evict_keys_that_no_cluster_holds():
    """More slots than the shared memory of sixteen CTAs has keys for: they are formed again for every pass."""
    rng = np.random.default_rng(31)
    run_evict(rng, [270001, 7], 1, 64, 128, 300, 2, 50, missing=[(0, 5), (0, 2000)])


def test_evict_reports_contradictions():
    p = C.make_kv_params(num_reqs=2, num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=16, max_seqlen=32, num_kv4_pages=6,
                         max_pages_per_req=2, budget=16, max_dst_pages=1)
    rng = np.random.default_rng(0)
    cache = noise_cache(rng, 6, 1, 16, 64)
    before = cache.clone()
    for bad in (33, -1):
        st = new_status()
        n, kept, w = C.cosa_kv4_evict(p, cache, i32([[0, 1], [2, 3]]), i32([bad, 0]), torch.ones(2, 1, 32, device=DEV),
                                      i32([[4], [5]]), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == cosa.COSA_ERR_BAD_INPUT and n.tolist() == [0, 0] and (kept == -1).all()
    assert torch.equal(cache, before)
