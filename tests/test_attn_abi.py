"""libcosa_attn loads without a GPU, exports what include/cosa_attn.h declares, and refuses bad arguments on the host."""
import copy
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WS = -1, -2, -5


@pytest.fixture(scope="module")
def C():
    from block_sparse_long_gb300 import build
    build.build()
    from block_sparse_long_gb300 import attn
    return attn


def header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "cosa_attn.h")).read(), flags=re.S)


def test_exports(C):
    out = subprocess.run(["nm", "-D", "--defined-only", C.ATTN_LIB_PATH], capture_output=True, text=True).stdout
    declared = set(re.findall(r"\b(cosa_\w+)\s*\(", header()))
    assert set(re.findall(r" T (cosa_\w+)", out)) == declared == set(C.ATTN_EXPORTS)
    out = subprocess.run(["ldd", C.ATTN_LIB_PATH], capture_output=True, text=True).stdout
    assert "libcuda.so" not in out and "libcudart" not in out
    assert C.cosa_attn_version() >= 1


def test_params_mirror_the_header(C):
    """Field by field, in order, with the header's types."""
    text = header()
    body = text[text.index("typedef struct cosa_attn_params {"):text.index("} cosa_attn_params;")]
    fields = re.findall(r"(int32_t|int64_t|double)\s+(\w+);", body)
    types = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "double": ctypes.c_double}
    assert [(n, types[t]) for t, n in fields] == list(C.CosaAttnParams._fields_)
    assert int(re.search(r"COSA_ATTN_ROPE_DIM (\d+)", text)[1]) == C.COSA_ATTN_ROPE_DIM
    assert int(re.search(r"COSA_ATTN_MAX_TREE (\d+)", text)[1]) == C.COSA_ATTN_MAX_TREE
    assert int(re.search(r"COSA_ATTN_FLAG_INTERLEAVED (\d+)", text)[1]) == C.COSA_ATTN_FLAG_INTERLEAVED
    assert int(re.search(r"COSA_ATTN_FLAG_TEST_STALL (\d+)", text)[1]) == C.COSA_ATTN_FLAG_TEST_STALL


F = ctypes.c_void_p(4096)          # an aligned address that no refused call looks at
G = ctypes.c_void_p(8192)
ODD = ctypes.c_void_p(4104)        # not 16-byte aligned


def params(C, **kw):
    base = dict(num_reqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, latent_dim=512, page_size=64, total_tokens=10, total_kv_tokens=20,
                max_seqlen=1000, num_pages=40, max_pages_per_req=16, max_new_tokens=8)
    later = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride") or k in ("flags", "reserved", "sm_scale")}
    base.update(kw)
    p = C.make_attn_params(**base)
    for k, v in later.items():
        setattr(p, k, v)
    return p


def tree(C, p, q=F, k=F, v=F, pt=F, n=F, cu=F, mask=F, out=G, lse=F, ws=F, size=1 << 40):
    return C.attn_library().cosa_tree_attention(ctypes.byref(p), q, cu, k, v, pt, n, mask, out, lse, ws, size, None, None)


def latent(C, p, q=F, qr=F, k=F, pt=F, n=F, cu=F, mask=F, out=G, lse=F, ws=F, size=1 << 40):
    return C.attn_library().cosa_latent_attention(ctypes.byref(p), q, qr, cu, k, pt, n, mask, out, lse, ws, size, None, None)


def commit(C, p, a=F, b=G, row=256, cu=F, pt=F, n=F, path=F, m=F, new=G):
    return C.attn_library().cosa_tree_commit(ctypes.byref(p), a, b, row, cu, pt, n, path, m, new, None, None)


def rope(C, p, kv=F, q=F, w=F, inv=F, cu=F, q_out=G, c=G, k=G, cache=G, pt=F):
    return C.attn_library().cosa_latent_rope(ctypes.byref(p), kv, q, w, inv, None, cu, None, q_out, c, k, cache, pt, None, None)


def prefill(C, p, q=F, qr=F, k=F, kr=F, v=F, cu=F, cu_kv=F, out=G, lse=F):
    return C.attn_library().cosa_latent_prefill(ctypes.byref(p), q, qr, k, kr, v, cu, cu_kv, out, lse, None, None)


PAGED = (tree, latent, commit, rope)
ATTENTIONS = (tree, latent, prefill)


def test_parameters_refused(C):
    for kw, code in ((dict(num_reqs=0), INV), (dict(num_q_heads=0), INV), (dict(total_tokens=-1), INV), (dict(flags=2), INV), (dict(reserved=1), INV),
                     (dict(num_reqs=70000), UNS), (dict(num_q_heads=1 << 17), UNS), (dict(total_tokens=(1 << 30) + 1), UNS)):
        for call in (*PAGED, prefill):
            assert call(C, params(C, **kw)) == code, (kw, call)
    for kw, code in ((dict(max_seqlen=0), INV), (dict(max_pages_per_req=15), INV), (dict(num_pages=0), INV), (dict(page_size=48), UNS),
                     (dict(page_size=256), UNS), (dict(num_pages=1 << 25, page_size=64), UNS),
                     (dict(max_seqlen=(1 << 30) + 1, max_pages_per_req=1 << 25), UNS)):
        for call in PAGED:
            assert call(C, params(C, **kw)) == code, (kw, call)
        assert C.cosa_tree_attention_workspace_size(params(C, **kw)) == C.cosa_latent_attention_workspace_size(params(C, **kw)) == 0
    for kw in (dict(sm_scale=0.0), dict(sm_scale=-1.0), dict(sm_scale=float("nan")), dict(sm_scale=1e30), dict(max_new_tokens=0), dict(q_stride=8),
               dict(q_stride=8 * 512 + 4)):
        for call in ATTENTIONS:
            assert call(C, params(C, **kw)) == INV, (kw, call)
    head_major = dict(q_stride=512, q_head_stride=512 * 10)        # ten tokens within a head
    assert C.cosa_latent_attention_workspace_size(params(C, **head_major)) > 0
    assert latent(C, params(C, q_stride=512, q_head_stride=512 * 9)) == INV
    for kw, code in ((dict(num_kv_heads=0), INV), (dict(num_kv_heads=3), INV), (dict(head_dim=96), UNS), (dict(head_dim=192), UNS)):
        assert tree(C, params(C, **kw)) == code
    for kw in (dict(latent_dim=128), dict(latent_dim=0), dict(latent_dim=640)):
        assert latent(C, params(C, **kw)) == rope(C, params(C, **kw)) == UNS
    for kw, code in ((dict(head_dim=192), UNS), (dict(total_kv_tokens=-1), INV), (dict(total_kv_tokens=0), INV), (dict(total_kv_tokens=(1 << 30) + 1), UNS),
                     (dict(k_stride=1000), INV), (dict(k_head_stride=64), INV), (dict(v_stride=1028), INV), (dict(v_head_stride=132), INV),
                     (dict(q_rope_stride=500), INV), (dict(q_rope_head_stride=32), INV), (dict(k_rope_stride=32), INV), (dict(q_head_stride=1 << 33), INV)):
        assert prefill(C, params(C, **kw)) == code, kw
    assert latent(C, params(C, q_rope_stride=500)) == INV
    many = dict(num_reqs=60000, total_tokens=60000, max_seqlen=1 << 23, max_pages_per_req=1 << 17)     # more tiles than 31 bits number
    assert tree(C, params(C, **many)) == latent(C, params(C, **many)) == UNS
    assert C.cosa_tree_attention_workspace_size(params(C, **many)) == 0
    for call in ATTENTIONS:
        assert call(C, params(C, num_q_heads=1 << 14, total_tokens=1 << 18)) == UNS


def test_prefill_of_more_blocks_than_a_grid_has(C):
    """Blocks of 128 queries, one at least for a request, times heads: what a launch cannot number is refused as such."""
    for kw in (dict(num_reqs=60000, num_q_heads=60000, total_tokens=10), dict(num_reqs=65535, num_q_heads=32769, total_tokens=65535)):
        assert prefill(C, params(C, **kw)) == UNS
    assert prefill(C, params(C, num_reqs=60000, num_q_heads=30000, total_tokens=0)) == 0


def test_fields_without_use_are_ignored(C):
    """What the header says of them, on calls without tokens, which do nothing."""
    slots = dict(page_size=3, max_seqlen=0, num_pages=0, max_pages_per_req=0)
    for call, junk in ((tree, dict(latent_dim=7, total_kv_tokens=-1, norm_eps=-1.0)), (latent, dict(num_kv_heads=0, head_dim=1, total_kv_tokens=-1)),
                       (prefill, dict(slots, num_kv_heads=0, latent_dim=7, norm_eps=-1.0)),
                       (rope, dict(num_kv_heads=0, head_dim=1, total_kv_tokens=-1, max_new_tokens=0, sm_scale=0.0))):
        assert call(C, params(C, total_tokens=0, **junk)) == 0, call
    assert rope(C, params(C, total_tokens=0, **slots), cache=None, pt=None) == 0


def test_attention_arguments_refused(C):
    p = params(C)
    for call, names in ((tree, ("q", "k", "v", "pt", "n", "cu", "out")), (latent, ("q", "qr", "k", "pt", "n", "cu", "out")),
                        (prefill, ("q", "qr", "k", "kr", "v", "cu", "out"))):
        for name in names:
            assert call(C, p, **{name: None}) == INV, (call, name)
        for name in ("q", "k", "out") + (("v",) if call is not latent else ("qr",)):
            assert call(C, p, **{name: ODD}) == INV, (call, name)
        assert call(C, p, q=G) == INV                                   # out is q
        assert call(C, p, lse=ctypes.c_void_p(4097)) == INV
        assert call(C, params(C, total_tokens=0), q=None) == 0          # nothing to do
    for call, size in ((tree, C.cosa_tree_attention_workspace_size(p)), (latent, C.cosa_latent_attention_workspace_size(p))):
        assert size > 0
        assert call(C, p, ws=None) == call(C, p, ws=ODD) == call(C, p, size=size - 1) == WS
        assert call(C, p, mask=ctypes.c_void_p(4100)) == INV
    for name in ("k", "v", "kr", "qr"):
        assert prefill(C, p, **{name: G}) == INV                        # out is an input


def test_outputs_that_other_ctas_still_read(C):
    H = ctypes.c_void_p(16384)
    assert latent(C, params(C), qr=G) == INV                             # out is q_rope
    for name in ("cu", "pt", "n", "path", "m"):
        assert commit(C, params(C), **{name: H}, new=H) == INV           # new_len is an input


def test_commit_arguments_refused(C):
    p = params(C)
    for name in ("a", "cu", "pt", "n", "path", "m", "new"):
        assert commit(C, p, **{name: None}) == INV
    for kw in (dict(row=0), dict(row=12), dict(row=-8), dict(a=ODD), dict(b=ODD), dict(new=F), dict(a=F, b=F)):
        assert commit(C, p, **kw) == INV, kw
    assert commit(C, p, row=1 << 23) == commit(C, params(C, max_new_tokens=65)) == UNS
    assert commit(C, params(C, max_new_tokens=0)) == INV


def test_rope_arguments_refused(C):
    p = params(C)
    for kw in (dict(kv=None), dict(inv=None), dict(cu=None), dict(q_out=None), dict(q=None), dict(c=None), dict(k=None), dict(cache=None),
               dict(pt=None), dict(c=None, k=None, cache=None, pt=None), dict(kv=ODD), dict(q=ODD), dict(w=ODD), dict(cache=ODD),
               dict(inv=ctypes.c_void_p(4100)), dict(c=F), dict(cache=F)):
        assert rope(C, p, **kw) == INV, kw
    for kw in (dict(k_stride=500), dict(k_stride=580), dict(q_rope_stride=500), dict(q_rope_head_stride=60), dict(q_rope_head_stride=68)):
        assert rope(C, params(C, **kw)) == INV, kw
    for eps in (-1.0, float("nan"), float("inf"), 1e-40, 1e300):
        assert rope(C, params(C, norm_eps=eps)) == INV, eps
    # in place needs dense rows
    assert rope(C, params(C, q_rope_head_stride=192), q_out=F) == rope(C, params(C, q_rope_stride=1024), q_out=F) == INV
    assert rope(C, params(C, total_tokens=0), kv=None) == 0


def test_binding_refuses_what_does_not_fit(C):
    """The binding looks at types and shapes before it looks for a device."""
    p = params(C)
    q, cu, pt, n = torch.zeros(10, 8, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 16, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    kc = torch.zeros(40, 64, 2, 128, dtype=torch.bfloat16)
    for bad in (q.float(), q[:9], q[:, :7], q.transpose(1, 2).contiguous().transpose(1, 2), q[:1].expand(10, -1, -1), q):
        with pytest.raises(ValueError):
            C.cosa_tree_attention(p, bad, cu, kc, kc, pt, n)
    with pytest.raises(ValueError, match="one or two"):
        C.cosa_tree_commit(p, (), cu, pt, n, cu, n)
    with pytest.raises(ValueError, match="equal rows"):
        C.cosa_tree_commit(p, (kc, kc[:, :, :1].contiguous()), cu, pt, n, cu, n)
    with pytest.raises(ValueError, match="kv must be"):
        C.cosa_latent_rope(p, torch.zeros(10, 512, dtype=torch.bfloat16), cu, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="apart"):
        C.cosa_latent_rope(p, torch.zeros(1, 576, dtype=torch.bfloat16).expand(10, -1), cu, torch.zeros(32, dtype=torch.float64))


def test_sizes(C):
    p = params(C)
    need = C.attn_required_numel(p)
    assert need["out"] == 10 * 8 * 128 and need["latent_out"] == 10 * 8 * 512 and need["k_cache"] == 40 * 64 * 2 * 128
    assert need["latent_cache"] == 40 * 64 * 576 and need["path"] == 16 and need["lse"] == 80 and need["page_table"] == 32
    assert C.latent_cache_shape(3, 16, 256) == (3, 16, 320)


def test_latent_attention_refuses_the_default_scale(C):
    """It is the tree attention's, 1/sqrt(head_dim): a copy of the parameters has it too, one that was set does not."""
    given = params(C)
    assert not given.scale_given and given.sm_scale == pytest.approx(128 ** -0.5)
    q, r, cu, pt, n = torch.zeros(10, 8, 128, dtype=torch.bfloat16), torch.zeros(10, 8, 64, dtype=torch.bfloat16), *(torch.zeros(40, dtype=torch.int32) for _ in range(3))
    for p in (given, C.CosaAttnParams.from_buffer_copy(given), copy.copy(given)):
        with pytest.raises(ValueError, match="sm_scale"):
            C.cosa_latent_attention(p, q, r, cu, q, pt, n)
        with pytest.raises(ValueError, match="sm_scale"):
            C.cosa_latent_prefill(p, q, r, q, r[:, 0], q, cu)
    for p in (params(C, sm_scale=192 ** -0.5), C.make_attn_params(num_reqs=1, num_q_heads=1, sm_scale=128 ** -0.5)):
        for p in (p, C.CosaAttnParams.from_buffer_copy(p), copy.copy(p)):
            assert p.scale_given
            with pytest.raises(ValueError, match="q_latent must be|must be a CUDA"):
                C.cosa_latent_attention(p, q, r, cu, q, pt, n)
