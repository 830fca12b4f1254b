"""The calls of include/cosa_kv.h together and as a serving program makes them: after a sparse prefill, step by step with
an append, on streams of their own, captured into graphs, two at a time, and with the binding's refusals."""
import math

import numpy as np
import pytest
import torch

import synth
from block_sparse_long_gb300 import cosa, kv as C
from oracle import cosa_oracle as orc
from tests import gpu_helpers as gh, kv_reference as ref
from tests.kv_helpers import bf, cu_of, i32, new_status, ok, packed, table

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_sparse_long_gb300 import build
    build.build()


class Loop:
    """One layer's state: a prompt of two requests (heads 4 over 2), and everything a step writes."""

    def __init__(self, seed, lens=(150, 61), new=6, Hq=4, Hkv=2, d=64, P=16, budget=80):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.d, self.P, self.budget = list(lens), Hq, Hkv, d, P, budget
        B, T = len(lens), sum(lens)
        self.pages = -(-(max(lens) + new) // P)
        self.room = -(-(budget + new) // P)
        total = B * (self.pages + self.room)
        t = table(rng, B, self.pages + self.room, total)
        self.pt4, self.dst = np.ascontiguousarray(t[:, :self.pages]), np.ascontiguousarray(t[:, self.pages:])
        self.pt = table(rng, B, self.pages, B * self.pages)
        self.common = dict(num_reqs=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, page_size=P, max_seqlen=self.pages * P,
                           num_pages=B * self.pages, num_kv4_pages=total, max_pages_per_req=self.pages, rotary_dim=d,
                           budget=budget, sink=2, recent=8, max_dst_pages=self.room)
        self.p = C.make_kv_params(total_tokens=T, **self.common)
        self.p1 = C.make_kv_params(total_tokens=B, **self.common)
        self.inv = torch.from_numpy(1e4 ** (-np.arange(d // 2) / (d // 2))).to(DEV)
        self.qkv = bf(rng, T, Hq + 2 * Hkv, d)
        self.steps = [bf(rng, B, Hq + 2 * Hkv, d) for _ in range(new)]
        self.wq, self.wk = bf(rng, d) * 0.1 + 1, bf(rng, d) * 0.1 + 1
        self.cache = torch.zeros(C.kv4_cache_shape(total, Hkv, P, d), dtype=torch.uint8, device=DEV)
        self.kc, self.vc = (torch.zeros(B * self.pages, P, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.weights = torch.zeros(B, Hkv, self.pages * P, device=DEV)
        self.kv_len = i32(self.lens)
        self.pos = list(self.lens)
        self.status = new_status()

    def split(self, x):
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def prefill(self):
        q, k, v = self.split(self.qkv)
        q_out, _ = C.cosa_qk_norm_rope(self.p, q, k, cu_of(self.lens), self.inv, v=v, q_weight=self.wq, k_weight=self.wk,
                                       k_cache=self.kc, v_cache=self.vc, page_table=i32(self.pt), status=self.status)
        C.cosa_kv4_store(self.p, self.cache, i32(self.pt4), self.kc, self.vc, src_page_table=i32(self.pt), kv_len=self.kv_len,
                         status=self.status)
        return q_out

    def step(self, n, table4):
        """Decode of one token per request."""
        q, k, v = self.split(self.steps[n])
        B = len(self.lens)
        q1, k1 = C.cosa_qk_norm_rope(self.p1, q, k, cu_of([1] * B), self.inv, q_weight=self.wq, k_weight=self.wk,
                                     positions=i32(self.pos), status=self.status)
        C.cosa_kv4_store(self.p1, self.cache, table4, k1, v, cu_seqlens=cu_of([1] * B), start=self.kv_len, status=self.status)
        self.kv_len = self.kv_len + 1
        self.pos = [x + 1 for x in self.pos]
        return C.cosa_kv4_attention(self.p1, q1, cu_of([1] * B), self.cache, table4, self.kv_len, weights=self.weights, status=self.status)


def test_prefill_decode_evict_reload():
    """Norm and rotation feed the proxy and the sparse prefill (with every block selected: dense causal attention); the pages go
    to 4 bits; decode steps append and attend; the cache is thinned and decoding goes on; the thinned cache goes back to
    bf16.  Each against a float64 run of the same chain from the same bf16 values."""
    s = Loop(1)
    q_out = s.prefill()
    ok(s.status)
    B, d, P, g = 2, s.d, s.P, s.Hq // s.Hkv
    scale = 1 / math.sqrt(d)

    # the prefill's own calls on what the new call wrote
    L = max(s.lens)
    p = cosa.params_for(q_out, s.kc, i32(s.pt), cu_of(s.lens), block_size=64, max_seqlen=L, stride=8)
    mask, mask_len = cosa.cosa_proxy_select(p, q_out, cu_of(s.lens), s.kc, i32(s.pt), status=s.status)
    out = cosa.cosa_sparse_prefill(p, q_out, cu_of(s.lens), s.kc, s.vc, i32(s.pt), mask, mask_len, status=s.status)
    ok(s.status)
    k16, v16, q16 = ref.to_f64(s.kc), ref.to_f64(s.vc), ref.to_f64(q_out)
    ks, vs, row = [], [], 0
    for b, n in enumerate(s.lens):
        at = [(int(s.pt[b, t // P]), t % P) for t in range(n)]
        k = np.stack([k16[a, z] for a, z in at])
        v = np.stack([v16[a, z] for a, z in at])
        want, mag, _ = ref.attention(q16[row:row + n], k, v, np.ones(n, bool), scale)
        assert np.abs(ref.to_f64(out[row:row + n]) - want).max() <= gh.O_MAX_ABS
        ks.append(ref.rounded(k))
        vs.append(ref.rounded(v))
        row += n

    # decode: three steps, thin, three more
    acc = [np.zeros((s.Hkv, n)) for n in s.lens]
    tab = i32(s.pt4)
    for n in range(6):
        if n == 3:
            kept_want = [[ref.evict(ref.to_f64(s.weights[b, h])[:len(ks[b])].astype(np.float32), np.ones(len(ks[b]), bool), s.budget, 2, 8)
                          for h in range(s.Hkv)] for b in range(B)]
            new_len, kept, s.weights = C.cosa_kv4_evict(s.p, s.cache, tab, s.kv_len, s.weights, i32(s.dst), status=s.status)
            ok(s.status)
            for b in range(B):
                for h in range(s.Hkv):
                    assert kept[b, h][:int(new_len[b])].tolist() == kept_want[b][h].tolist()
                m = len(kept_want[b][0])
                ks[b] = np.stack([ks[b][kept_want[b][h], h] for h in range(s.Hkv)], 1)
                vs[b] = np.stack([vs[b][kept_want[b][h], h] for h in range(s.Hkv)], 1)
                acc[b] = np.stack([acc[b][h][kept_want[b][h]] for h in range(s.Hkv)])
                assert m == int(new_len[b])
            s.kv_len = new_len
            # the destination pages are the first of a table as wide as the old one
            wide = np.full_like(s.pt4, -1)
            wide[:, :s.room] = s.dst
            tab = i32(wide)
        pos = list(s.pos)
        out = s.step(n, tab)
        ok(s.status)
        q, k, v = (ref.to_f64(x) for x in s.split(s.steps[n]))
        w = [ref.to_f64(x) for x in (s.wq, s.wk)]
        inv = s.inv.cpu().numpy()
        q1 = ref.bf16(ref.norm_rope(q, w[0], np.array(pos), inv, False, 1e-6)[0])
        k1 = ref.bf16(ref.norm_rope(k, w[1], np.array(pos), inv, False, 1e-6)[0])
        for b in range(B):
            # a key or query one fp32 rounding from a border may round to the neighbouring bf16: 2^-7 of it, as may the
            # 4-bit code of such a key (a step of the scale, at most 1/7 of the largest value of its group); the new key
            # is read back from the cache instead of assumed, within one step of the reference's
            got_k, got_v, _ = ref.unpack_request(s.cache.cpu().numpy(), tab[b].cpu().numpy(), len(ks[b]) + 1, d)
            step = np.abs(k1[b]).reshape(s.Hkv, -1, 32).max(-1) / 7 * 1.02
            assert (np.abs(got_k[-1] - ref.rounded(k1[b])).reshape(s.Hkv, -1, 32).max(-1) <= step).all()
            assert np.array_equal(got_v[-1], ref.rounded(v[b]))
            ks[b] = np.concatenate([ks[b], got_k[-1:]])
            vs[b] = np.concatenate([vs[b], got_v[-1:]])
            assert np.array_equal(ks[b], got_k) and np.array_equal(vs[b], got_v)
            want, mag, prob = ref.attention(q1[b:b + 1], ks[b], vs[b], np.ones(len(ks[b]), bool), scale)
            # queries off by 2^-7 of their size: a logit by 2^-7 |q| |k| scale, in a few of the values; a quarter of that in all
            e = 2.0 ** -9 * (np.abs(q1[b]).sum(-1).max() * np.abs(ks[b]).max()) * scale + ref.logit_error(q1[b:b + 1], ks[b], scale)
            assert (np.abs(ref.to_f64(out[b:b + 1]) - want) <= np.abs(want) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -17 + 2.1 * e)).all()
            add = prob.reshape(1, s.Hkv, g, -1).sum((0, 2))
            acc[b] = np.concatenate([acc[b], np.zeros((s.Hkv, 1))], 1) + add
            assert (np.abs(ref.to_f64(s.weights[b, :, :len(ks[b])]) - acc[b]) <= acc[b] * (2.1 * e + 2.0 ** -17)).all()
    # and back to bf16 pages
    kb, vb = torch.zeros_like(s.kc), torch.zeros_like(s.vc)
    C.cosa_kv4_load(s.p, s.cache, tab, kb, vb, i32(s.pt), kv_len=s.kv_len, status=s.status)
    ok(s.status)
    kn, vn = ref.to_f64(kb), ref.to_f64(vb)
    for b in range(B):
        for t in range(len(ks[b])):
            assert np.array_equal(kn[int(s.pt[b, t // P]), t % P], ref.bf16(ks[b][t]))
            assert np.array_equal(vn[int(s.pt[b, t // P]), t % P], ref.bf16(vs[b][t]))


def calls(seed):
    """Each call once on inputs of its own: [(run(stream) -> list of outputs)], outputs in buffers that exist."""
    s = Loop(seed)
    s.prefill()
    torch.cuda.synchronize()
    B, T = 2, sum(s.lens)
    q, k, v = s.split(s.qkv)
    cu, pt, pt4, dst, lens, cu1 = cu_of(s.lens), i32(s.pt), i32(s.pt4), i32(s.dst), i32(s.lens), cu_of([1] * B)
    q1 = bf(s.rng, B, s.Hq, s.d)
    e = lambda *a, dtype=torch.bfloat16: torch.zeros(a, dtype=dtype, device=DEV)  # noqa: E731
    q_out, k_out, kc, vc, kb, vb = e(T, s.Hq, s.d), e(T, s.Hkv, s.d), torch.zeros_like(s.kc), torch.zeros_like(s.vc), torch.zeros_like(s.kc), torch.zeros_like(s.vc)
    c4, c5 = torch.zeros_like(s.cache), torch.zeros_like(s.cache)
    out, acc = e(B, s.Hq, s.d), torch.zeros_like(s.weights)
    w = torch.rand_like(s.weights)
    ws = torch.empty(C.cosa_kv4_attention_workspace_size(s.p1, True), dtype=torch.uint8, device=DEV)
    nl, kept, wo = e(B, dtype=torch.int32), e(B, s.Hkv, s.budget, dtype=torch.int32), torch.zeros_like(w)
    c6 = s.cache.clone()

    def rope(st):
        C.cosa_qk_norm_rope(s.p, q, k, cu, s.inv, v=v, q_weight=s.wq, k_weight=s.wk, q_out=q_out, k_out=k_out, k_cache=kc, v_cache=vc,
                            page_table=pt, stream=st)
        return [q_out, k_out, kc, vc]

    def store_rows(st):
        C.cosa_kv4_store(s.p, c4, pt4, k, v, cu_seqlens=cu, stream=st)
        return [c4]

    def store_pages(st):
        C.cosa_kv4_store(s.p, c5, pt4, s.kc, s.vc, src_page_table=pt, kv_len=lens, stream=st)
        return [c5]

    def load(st):
        C.cosa_kv4_load(s.p, s.cache, pt4, kb, vb, pt, kv_len=lens, stream=st)
        return [kb, vb]

    def attend(st):
        acc.zero_() if st is None else None
        C.cosa_kv4_attention(s.p1, q1, cu1, s.cache, pt4, lens, out=out, weights=acc, workspace=ws, stream=st)
        return [out, acc]

    def evict(st):
        C.cosa_kv4_evict(s.p, c6, pt4, lens, w, dst, new_len=nl, kept=kept, weights_out=wo, stream=st)
        return [nl, kept, wo, c6]

    return s, [rope, store_rows, store_pages, load, attend, evict]


NAMES = ("rope", "store_rows", "store_pages", "load", "attend", "evict")


def wipe(tensors, which):
    """What a call is to write, spoilt (an accumulator and a cache that is also read are only reset)."""
    for t in tensors:
        if which == "evict" and t.dtype == torch.uint8:
            continue
        t.zero_()


@pytest.mark.parametrize("which", NAMES)
def test_on_another_stream_and_captured(which):
    """The whole call runs on the stream that it is given, behind what that stream waits for, and nothing of it on
    another; captured into a graph it does the same at every replay."""
    _, runs = calls(7)
    run = runs[NAMES.index(which)]
    outs = run(None)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    assert any(bool((t != 0).any()) for t in want)

    side = torch.cuda.Stream()
    wipe(outs, which)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)        # the stream is busy for milliseconds: nothing may be written meanwhile
    run(side)
    marker = torch.cuda.Event()
    marker.record(side)
    early = [t.clone() for t in outs]        # on the current stream, at once
    torch.cuda.current_stream().synchronize()
    assert not marker.query(), "the side stream ended too soon for the check to mean anything"
    for t, w in zip(early, want):
        assert which == "evict" and t.dtype == torch.uint8 or not bool((t != 0).any())
    side.synchronize()
    assert all(torch.equal(t, w) for t, w in zip(outs, want))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(side)
    for _ in range(3):
        wipe(outs, which)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(outs, want))


def test_two_attentions_at_once():
    """Two calls on two streams, each with a workspace, many times: the results of each alone."""
    pairs = [calls(k)[1][4] for k in (11, 12)]
    want = []
    for run in pairs:
        outs = run(None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in pairs]
    buffers = [run(None) for run in pairs]
    for _ in range(20):
        for t in sum(buffers, []):
            t.zero_()
        torch.cuda.synchronize()
        for st, run in zip(streams, pairs):
            run(st)
        torch.cuda.synchronize()
        for outs, w in zip(buffers, want):
            assert all(torch.equal(t, x) for t, x in zip(outs, w))


def test_allocates_outputs_on_the_given_stream():
    """Outputs and workspace that the binding allocates belong to the call's stream: their memory is not handed out again
    while the call may still use it."""
    s, _ = calls(13)
    side = torch.cuda.Stream()
    q1 = bf(s.rng, 2, s.Hq, s.d)
    args = (s.p1, q1, cu_of([1, 1]), s.cache, i32(s.pt4), i32(s.lens))
    want = C.cosa_kv4_attention(*args)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = C.cosa_kv4_attention(*args, stream=side)
    for _ in range(50):                       # what the current stream allocates now must not be the workspace
        torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_attention_on_a_batch_with_padding():
    """Graph-style padding: more requests than are alive (no queries, length 0), more rows than cu_seqlens covers; the same
    results as without."""
    rng = np.random.default_rng(21)
    lens = [40, 33]
    cache, t, ks, vs = packed(rng, lens, 2, 16, 64)
    q = bf(rng, 8, 4, 64)
    small = C.make_kv_params(num_reqs=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, total_tokens=2, max_seqlen=48,
                             num_kv4_pages=cache.shape[0], max_pages_per_req=3)
    want = C.cosa_kv4_attention(small, q[:2].contiguous(), cu_of([1, 1]), cache, i32(t), i32(lens))
    big = C.make_kv_params(num_reqs=5, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, total_tokens=8, max_seqlen=48,
                           num_kv4_pages=cache.shape[0], max_pages_per_req=3)
    t5 = np.full((5, 3), -1, np.int32)
    t5[[0, 3]] = t
    out = bf(rng, 8, 4, 64)
    guard = out.clone()
    C.cosa_kv4_attention(big, q, i32([0, 1, 1, 1, 2, 2]), cache, i32(t5), i32([40, 0, 0, 33, 0]), out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[:2], want) and torch.equal(out[2:], guard[2:])


def test_shared_prefix_pages_are_read_by_both():
    """Two requests whose tables share pages (a common prompt): each reads them."""
    rng = np.random.default_rng(22)
    cache, t, ks, vs = packed(rng, [64], 2, 16, 64)
    q = bf(rng, 2, 4, 64)
    p = C.make_kv_params(num_reqs=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, total_tokens=2, max_seqlen=64,
                         num_kv4_pages=cache.shape[0], max_pages_per_req=4)
    out = C.cosa_kv4_attention(p, torch.cat([q[:1], q[:1]]), cu_of([1, 1]), cache, i32(np.concatenate([t, t])), i32([64, 64]))
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1])


def test_pages_beyond_32_bits():
    """Caches of more than 2^32 bytes whose used pages are the last ones: every call gives what it gives on small caches."""
    H, d, P, lens = 8, 128, 64, [130, 65]
    rng = np.random.default_rng(33)
    near, pages, room = 12, 3, 2
    far16 = (1 << 32) // (P * H * d * 2) + 100          # bf16 pages: 4 GiB and some
    far4 = (1 << 32) // (P * H * d * 9 // 8) + 100
    T = sum(lens)
    qkv = bf(rng, T, 4 * H + 2 * H, d)
    inv = torch.from_numpy(1e4 ** (-np.arange(d // 2) / (d // 2))).to(DEV)
    w = torch.rand(2, H, pages * P, device=DEV)
    t16, t4 = table(rng, 2, pages, near), table(rng, 2, pages + room, near)
    q1 = bf(rng, 2, 4 * H, d)
    got = []
    for n16, n4 in ((near, near), (far16, far4)):
        a, b = t16 + (n16 - near), t4 + (n4 - near)
        src, dst = i32(np.ascontiguousarray(b[:, :pages])), i32(np.ascontiguousarray(b[:, pages:]))
        kw = dict(num_reqs=2, num_q_heads=4 * H, num_kv_heads=H, head_dim=d, page_size=P, max_seqlen=pages * P, num_pages=n16,
                  num_kv4_pages=n4, max_pages_per_req=pages, budget=100, sink=1, recent=9, max_dst_pages=room)
        p = C.make_kv_params(total_tokens=T, **kw)
        kc, vc = (torch.zeros(n16, P, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        cache = torch.zeros(C.kv4_cache_shape(n4, H, P, d), dtype=torch.uint8, device=DEV)
        st = new_status()
        q_out, _ = C.cosa_qk_norm_rope(p, qkv[:, :4 * H], qkv[:, 4 * H:5 * H], cu_of(lens), inv, v=qkv[:, 5 * H:], k_cache=kc,
                                       v_cache=vc, page_table=i32(a), status=st)
        C.cosa_kv4_store(p, cache, src, kc, vc, src_page_table=i32(a), kv_len=i32(lens), status=st)
        C.cosa_kv4_store(p, cache, src, qkv[:, 4 * H:5 * H], qkv[:, 5 * H:], cu_seqlens=i32([0, 1, 2]), start=i32([7, 64]), status=st)
        acc = w.clone()
        out = C.cosa_kv4_attention(C.make_kv_params(total_tokens=2, **kw), q1, cu_of([1, 1]), cache, src, i32(lens), weights=acc, status=st)
        new_len, kept, wo = C.cosa_kv4_evict(p, cache, src, i32(lens), w, dst, status=st)
        kb, vb = torch.zeros_like(kc), torch.zeros_like(vc)
        C.cosa_kv4_load(C.make_kv_params(**{**kw, "max_seqlen": room * P, "max_pages_per_req": room}), cache, dst, kb, vb,
                        i32(np.ascontiguousarray(a[:, :room])), kv_len=new_len, status=st)
        ok(st)
        got.append([q_out, out, acc, new_len, kept, wo, kc[n16 - near:], vc[n16 - near:], cache[n4 - near:], kb[n16 - near:], vb[n16 - near:]])
        if n16 > near:
            assert not bool(kc[:n16 - near].any()) and not bool(cache[:n4 - near].any()) and not bool(vb[:n16 - near].any())
        got[-1] = [x.clone() for x in got[-1]]
        del kc, vc, cache, kb, vb
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert bool(got[0][-1].any()) and bool(got[0][1].any())


def test_waits_that_run_out_end_the_kernel():
    """With no copy issued, every wait of the attention runs out: the call ends by itself and reports it, and the next call is
    as good as ever."""
    s, _ = calls(15)
    q1 = bf(s.rng, 2, s.Hq, s.d)
    args = (q1, cu_of([1, 1]), s.cache, i32(s.pt4), i32(s.lens))
    want = C.cosa_kv4_attention(s.p1, *args)
    torch.cuda.synchronize()
    p = C.CosaKvParams.from_buffer_copy(s.p1)
    p.flags |= C.COSA_KV_FLAG_TEST_STALL
    st = new_status()
    C.cosa_kv4_attention(p, *args, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == cosa.COSA_ERR_DEVICE_TIMEOUT
    st = new_status()
    assert torch.equal(C.cosa_kv4_attention(s.p1, *args, status=st), want)
    ok(st)


def test_binding_refusals_on_the_device():
    s, _ = calls(14)
    ok_args = dict(cu=cu_of([1, 1]), pt=i32(s.pt4), lens=i32(s.lens))
    q1 = bf(s.rng, 2, s.Hq, s.d)
    with pytest.raises(ValueError, match="kv_len"):
        C.cosa_kv4_attention(s.p1, q1, ok_args["cu"], s.cache, ok_args["pt"], i32([3]))
    with pytest.raises(ValueError, match="page_table"):
        C.cosa_kv4_attention(s.p1, q1, ok_args["cu"], s.cache, ok_args["pt"].long(), ok_args["lens"])
    with pytest.raises(ValueError, match="kv4_cache"):
        C.cosa_kv4_attention(s.p1, q1, ok_args["cu"], s.cache[:-1], ok_args["pt"], ok_args["lens"])
    with pytest.raises(cosa.CosaError, match="workspace"):
        C.cosa_kv4_attention(s.p1, q1, ok_args["cu"], s.cache, ok_args["pt"], ok_args["lens"],
                             workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(cosa.CosaError, match="unsupported"):
        C.cosa_kv4_attention(s.p1, bf(s.rng, 2, 2 * s.Hq, s.d)[:, :s.Hq], ok_args["cu"], s.cache, ok_args["pt"], ok_args["lens"])
    with pytest.raises(ValueError, match="status"):
        C.cosa_kv4_attention(s.p1, q1, ok_args["cu"], s.cache, ok_args["pt"], ok_args["lens"], status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(cosa.CosaError, match="invalid"):
        C.cosa_kv4_evict(s.p, s.cache, ok_args["pt"], ok_args["lens"], s.weights, ok_args["pt"])
