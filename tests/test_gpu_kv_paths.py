"""The calls of include/cosa_kv.h on the paths that small shapes do not reach: the attention's list of the whole batch with its
join, whichever way its waits end, long contexts, many rows."""
import time

import numpy as np
import pytest
import torch

from block_sparse_long_gb300 import cosa, kv as C
from tests import kv_paths, test_gpu_kv as base
from tests.kv_helpers import cu_of, i32, new_status, ok

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
