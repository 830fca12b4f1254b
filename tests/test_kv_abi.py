"""libcosa_kv loads without a GPU, exports what include/cosa_kv.h declares, and refuses bad arguments on the host."""
import ctypes
import os
import re
import subprocess
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def C():
    from block_sparse_long_gb300 import build
    build.build()
    from block_sparse_long_gb300 import kv
    return kv


def declared():
    text = open(os.path.join(ROOT, "include", "cosa_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return set(re.findall(r"\b(cosa_\w+)\s*\(", text))


def test_exports(C):
    out = subprocess.run(["nm", "-D", "--defined-only", C.KV_LIB_PATH], capture_output=True, text=True).stdout
    assert set(re.findall(r" T (cosa_\w+)", out)) == declared() == set(C.KV_EXPORTS)
    out = subprocess.run(["ldd", C.KV_LIB_PATH], capture_output=True, text=True).stdout
    assert "libcuda.so" not in out and "libcudart" not in out
    assert C.cosa_kv_version() >= 1


def test_params_mirror_the_header(C):
    """Field by field, in order, with the header's types."""
    text = open(os.path.join(ROOT, "include", "cosa_kv.h")).read()
    body = re.sub(r"/\*.*?\*/", "", text[text.index("typedef struct cosa_kv_params {"):text.index("} cosa_kv_params;")], flags=re.S)
    fields = re.findall(r"(int32_t|int64_t|double)\s+(\w+);", body)
    types = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "double": ctypes.c_double}
    assert [(n, types[t]) for t, n in fields] == list(C.CosaKvParams._fields_)


F = ctypes.c_void_p(4096)          # an aligned address that no refused call looks at
ODD = ctypes.c_void_p(4104)        # not 16-byte aligned


def params(C, **kw):
    base = dict(num_reqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=64, total_tokens=10, max_seqlen=1000,
                num_pages=40, num_kv4_pages=40, max_pages_per_req=16, budget=100, sink=4, recent=10, max_dst_pages=2)
    stride = {k: kw.pop(k) for k in list(kw) if k.endswith("_stride")}
    flags = kw.pop("flags", None)
    base.update(kw)
    p = C.make_kv_params(**base)
    for k, v in stride.items():
        setattr(p, k, v)
    if flags is not None:
        p.flags = flags
    return p


def rope(C, p, q=F, k=F, v=F, q_out=F, k_out=None, kc=F, vc=F, pt=F, qw=F, inv=F, cu=F):
    return C.kv_library().cosa_qk_norm_rope(ctypes.byref(p), q, k, v, qw, F, inv, None, cu, None, q_out, k_out, kc, vc, pt, None, None)


def store(C, p, k=F, src=None, cu=F, n=None, c=F, pt=F):
    return C.kv_library().cosa_kv4_store(ctypes.byref(p), k, F, cu, src, None, n, c, pt, None, None)


def load(C, p, n=F, kc=F, c=F):
    return C.kv_library().cosa_kv4_load(ctypes.byref(p), c, F, None, n, kc, F, F, None, None)


def attend(C, p, q=F, w=None, ws=F, size=1 << 40, n=F, out=ctypes.c_void_p(8192)):
    return C.kv_library().cosa_kv4_attention(ctypes.byref(p), q, F, F, F, n, out, w, ws, size, None, None)


def evict(C, p, w=F, dst=ctypes.c_void_p(8192), wout=None, n=F, kept=F, new=ctypes.c_void_p(8192)):
    return C.kv_library().cosa_kv4_evict(ctypes.byref(p), F, F, n, w, dst, new, kept, wout, None, None)


def test_parameters_refused_by_every_call(C):
    inv, uns = -1, -2
    for kw, code in ((dict(num_reqs=0), inv), (dict(num_q_heads=7), inv), (dict(num_kv_heads=0), inv),
                     (dict(head_dim=96), uns), (dict(page_size=48), uns), (dict(page_size=256), uns),
                     (dict(num_reqs=70000), uns), (dict(flags=2), inv)):
        p = params(C, **kw)
        for call in (rope, store, load, attend, evict):
            assert call(C, p) == code, (kw, call)
        assert C.cosa_kv4_attention_workspace_size(p) == 0
    for kw in (dict(max_seqlen=0), dict(max_pages_per_req=15), dict(max_pages_per_req=0), dict(num_kv4_pages=0)):
        for call in (store, load, attend, evict):
            assert call(C, params(C, **kw)) == inv, (kw, call)
    bad = params(C)
    bad.reserved = 1
    assert rope(C, bad) == inv
    assert rope(C, params(C, max_seqlen=1 << 30, max_pages_per_req=1 << 24, total_tokens=(1 << 30) + 1)) == uns


def test_rope_refusals(C):
    inv = -1
    for kw in (dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=144), dict(norm_eps=-1.0), dict(norm_eps=float("nan")),
               dict(norm_eps=float("inf")), dict(norm_eps=1e-40), dict(norm_eps=1e300), dict(total_tokens=-1), dict(q_stride=1023), dict(q_stride=1028), dict(k_stride=-256),
               dict(v_stride=8), dict(num_pages=0), dict(max_seqlen=0)):
        assert rope(C, params(C, **kw)) == inv, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(inv=None), dict(cu=None), dict(kc=None),
               dict(vc=None), dict(pt=None), dict(kc=None, vc=None, pt=None), dict(q=ODD), dict(qw=ODD), dict(kc=ODD)):
        assert rope(C, params(C), **kw) == inv, kw
    # in place needs dense rows
    assert rope(C, params(C, q_stride=2048), q_out=F) == inv
    assert rope(C, params(C, k_stride=2048), q=ctypes.c_void_p(8192), k_out=F) == inv
    assert rope(C, params(C, total_tokens=0), q=None) == 0          # nothing to do


def test_store_and_load_refusals(C):
    inv, uns = -1, -2
    p = params(C)
    for kw in (dict(k=None), dict(cu=None), dict(c=None), dict(pt=None), dict(k=ODD), dict(c=ODD), dict(src=F, n=None)):
        assert store(C, p, **kw) == inv, kw
    assert store(C, params(C, num_pages=0), src=F, n=F) == inv
    assert store(C, params(C, k_stride=2048), src=F, n=F) == uns     # pages are dense
    assert store(C, params(C, k_stride=12)) == inv
    assert store(C, params(C, total_tokens=-1)) == inv
    assert store(C, params(C, total_tokens=0), k=None) == 0
    for kw in (dict(n=None), dict(kc=None), dict(c=None), dict(kc=ODD)):
        assert load(C, p, **kw) == inv, kw
    assert load(C, params(C, num_pages=0)) == inv


def test_attention_refusals(C):
    inv, uns, wsp = -1, -2, -5
    for kw in (dict(sm_scale=0.0), dict(sm_scale=float("nan")), dict(sm_scale=1e-40), dict(sm_scale=1e30), dict(max_new_tokens=0), dict(total_tokens=-1)):
        assert attend(C, params(C, **kw)) == inv, kw
    assert attend(C, params(C, q_stride=2048)) == uns
    assert attend(C, params(C, total_tokens=1 << 30, num_q_heads=8, num_kv_heads=1)) == uns        # rows beyond 32 bits
    assert attend(C, params(C), q=None) == inv and attend(C, params(C), q=ODD) == inv and attend(C, params(C), n=None) == inv
    p = params(C)
    size = C.cosa_kv4_attention_workspace_size(p)
    more = C.cosa_kv4_attention_workspace_size(p, with_weights=True)
    assert 0 < size < more
    assert attend(C, p, size=size - 1) == wsp and attend(C, p, w=F, size=more - 1) == wsp
    assert attend(C, p, ws=None) == wsp and attend(C, p, ws=ctypes.c_void_p(4096 + 128)) == wsp
    assert attend(C, params(C, total_tokens=0), q=None) == 0
    assert attend(C, p, out=F) == inv                  # q itself


def test_evict_refusals(C):
    inv = -1
    for kw in (dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=60, recent=41), dict(max_dst_pages=1)):
        assert evict(C, params(C, **kw)) == inv, kw
    assert evict(C, params(C), w=None) == inv and evict(C, params(C), n=None) == inv and evict(C, params(C), kept=None) == inv
    assert evict(C, params(C), dst=F) == inv          # the source table
    assert evict(C, params(C), wout=F) == inv         # the weights themselves
    assert evict(C, params(C), new=F) == inv          # the old lengths


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_binding_refuses_before_the_library(C):
    """Sizes, types and layouts that the library cannot see.  Meta tensors stand for device memory: what passes every
    other check ends at the device check."""
    p = C.make_kv_params(num_reqs=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, total_tokens=6, max_seqlen=40,
                         num_pages=8, num_kv4_pages=9, max_pages_per_req=3, budget=20, max_dst_pages=2, rotary_dim=32)
    need = C.kv_required_numel(p)
    assert need["kv4_cache"] == 9 * 2 * 16 * 72 and need["k_cache"] == 8 * 16 * 2 * 64
    assert need["weights"] == 2 * 2 * 40 and need["kept"] == 2 * 2 * 20 and need["evict_page_table"] == 4
    assert need["page_table"] == 6 and need["inv_freq"] == 16 and need["q_out"] == 6 * 4 * 64
    assert C.kv4_cache_shape(9, 2, 16, 64) == (9, 2, 16, 72)
    c = C._Call(p)
    i32 = torch.int32
    with pytest.raises(ValueError, match="page_table holds 5"):
        c.dense((meta(5, dtype=i32), "page_table", i32))
    with pytest.raises(ValueError, match="must be torch.int32"):
        c.dense((meta(6, dtype=torch.int64), "page_table", i32))
    with pytest.raises(ValueError, match="contiguous"):
        c.dense((meta(6, 2, dtype=i32)[:, 0], "page_table", i32))
    with pytest.raises(ValueError, match="CUDA"):
        c.dense((meta(6, dtype=i32), "page_table", i32))
    with pytest.raises(ValueError, match="6"):
        c.rows(meta(5, 4, 64), "q", 4)
    with pytest.raises(ValueError, match="must be"):
        c.rows(meta(6, 256), "q", 4)
    with pytest.raises(ValueError, match="must be"):
        c.rows(meta(6, 4, 64, dtype=torch.float16), "q", 4)
    with pytest.raises(ValueError, match="heads of a token"):
        c.rows(meta(4, 6, 64).transpose(0, 1), "q", 4)
    with pytest.raises(ValueError, match="0 elements apart"):         # the library takes 0 for dense rows
        c.rows(meta(1, 4, 64).expand(6, 4, 64), "q", 4)
    with pytest.raises(ValueError, match="CUDA"):
        c.rows(meta(1, 4, 64).expand(6, 4, 64).contiguous(), "q", 4)
    with pytest.raises(ValueError, match="CUDA"):
        c.rows(meta(6, 8, 64)[:, :4], "q", 4)                         # a slice of a fused projection is fine
    c.index = 0
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        c.run("cosa_kv4_load", p, (), None, types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))
    with pytest.raises(ValueError, match="cu_seqlens"):
        C.cosa_kv4_store(p, None, None, None, None)
    with pytest.raises(ValueError, match="kv_len"):
        C.cosa_kv4_store(p, None, None, None, None, src_page_table=meta(6, dtype=i32))
