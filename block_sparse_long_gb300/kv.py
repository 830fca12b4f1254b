"""Thin Python binding of libcosa_kv's C ABI (include/cosa_kv.h): what stands around the sparse prefill.

Argument marshalling only, as in :mod:`block_sparse_long_gb300.cosa`: every step runs in the CUDA kernels
of libcosa_kv.so, PyTorch supplies device memory and streams, and there is no fallback.

The functions carry the C names:
  cosa_qk_norm_rope    norms of q and k per head, rotation, and the bf16 cache write (or k to rows)
  cosa_kv4_store       K and V, from rows or bf16 pages, into a paged 4-bit cache
  cosa_kv4_load        the 4-bit cache back into bf16 pages
  cosa_kv4_attention   attention of the newest tokens over the 4-bit cache, with accumulated weights
  cosa_kv4_evict       the slots with the largest accumulated weights moved into other pages
  cosa_kv4_attention_workspace_size, cosa_kv_version

A serving loop over one layer::

    p = make_kv_params(...)                                    # once per shape
    cosa_qk_norm_rope(p, q, k, cu, inv_freq, v=v, q_out=q_out, k_cache=k_cache, v_cache=v_cache, page_table=pt)
    # ... cosa_proxy_select and cosa_sparse_prefill on q_out and the pages ...
    cosa_kv4_store(p, kv4, pt4, k_cache, v_cache, src_page_table=pt, kv_len=kv_len)
    # decode, one token per request (kv_len counts it)
    q_out, k_out = cosa_qk_norm_rope(p1, q, k, cu1, inv_freq, positions=pos)
    cosa_kv4_store(p1, kv4, pt4, k_out, v, cu_seqlens=cu1, start=kv_len_before)
    out = cosa_kv4_attention(p1, q_out, cu1, kv4, pt4, kv_len, weights=weights)
    # when the cache is full
    new_len, kept, weights = cosa_kv4_evict(p, kv4, pt4, kv_len, weights, pt4_new)

Every call checks the tensors' types, sizes and device on the host, runs on the current stream of the
tensors' device (or ``stream``), and takes an optional int32 ``status`` tensor, zeroed by the caller, that
receives errors found on the device.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import torch

from .cosa import COSA_OK, CosaError

# Handle of the current stream of a device (the public way makes a Stream object for it, a microsecond per call).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)

_HERE = os.path.dirname(os.path.abspath(__file__))
KV_LIB_PATH = os.path.join(_HERE, "libcosa_kv.so")

# Every symbol include/cosa_kv.h declares.
KV_EXPORTS = ("cosa_kv_version", "cosa_qk_norm_rope", "cosa_kv4_store", "cosa_kv4_load",
              "cosa_kv4_attention_workspace_size", "cosa_kv4_attention", "cosa_kv4_evict")
COSA_KV_FLAG_INTERLEAVED = 1
COSA_KV_FLAG_TEST_STALL = 4   # test hook of cosa_kv4_attention: every in-kernel wait runs out
KV4_GROUP = 32   # values of a head that share a scale
KV4_TILE = 16    # tokens of a storage tile


class CosaKvParams(ctypes.Structure):
    """Mirror of ``cosa_kv_params``."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_reqs", "num_q_heads", "num_kv_heads", "head_dim", "page_size", "total_tokens", "max_seqlen", "num_pages",
        "num_kv4_pages", "max_pages_per_req", "rotary_dim", "max_new_tokens", "budget", "sink", "recent",
        "max_dst_pages", "flags", "reserved")] + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")] + [
        ("sm_scale", ctypes.c_double), ("norm_eps", ctypes.c_double)]


_lib = None


def kv_library() -> ctypes.CDLL:
    """Load libcosa_kv.so once.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(KV_LIB_PATH):
        raise RuntimeError(f"{KV_LIB_PATH} is missing: build it with `python -m block_sparse_long_gb300.build`")
    lib = ctypes.CDLL(KV_LIB_PATH)
    vp, sz, pp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(CosaKvParams)
    lib.cosa_kv_version.restype = ctypes.c_int
    lib.cosa_kv4_attention_workspace_size.restype = sz
    lib.cosa_kv4_attention_workspace_size.argtypes = [pp, ctypes.c_int]
    for name, pointers in (("cosa_qk_norm_rope", 15), ("cosa_kv4_store", 9), ("cosa_kv4_load", 8), ("cosa_kv4_evict", 9)):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [pp] + [vp] * (pointers + 1)
    lib.cosa_kv4_attention.restype = ctypes.c_int
    lib.cosa_kv4_attention.argtypes = [pp] + [vp] * 8 + [sz, vp, vp]
    _lib = lib
    return lib


def cosa_kv_version() -> int:
    return int(kv_library().cosa_kv_version())


def make_kv_params(*, num_reqs, num_q_heads, num_kv_heads, head_dim, page_size, total_tokens=0, max_seqlen=1,
                   num_pages=1, num_kv4_pages=1, max_pages_per_req=1, rotary_dim=None, interleaved=False,
                   max_new_tokens=1, budget=1, sink=0, recent=0, max_dst_pages=1, sm_scale=None,
                   norm_eps=1e-6) -> CosaKvParams:
    return CosaKvParams(
        num_reqs=num_reqs, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim, page_size=page_size,
        total_tokens=total_tokens, max_seqlen=max_seqlen, num_pages=num_pages, num_kv4_pages=num_kv4_pages,
        max_pages_per_req=max_pages_per_req, rotary_dim=head_dim if rotary_dim is None else rotary_dim,
        max_new_tokens=max_new_tokens, budget=budget, sink=sink, recent=recent, max_dst_pages=max_dst_pages,
        flags=COSA_KV_FLAG_INTERLEAVED if interleaved else 0,
        sm_scale=float(sm_scale if sm_scale is not None else 1.0 / math.sqrt(head_dim)), norm_eps=float(norm_eps))


def kv4_cache_shape(num_kv4_pages: int, num_kv_heads: int, page_size: int, head_dim: int) -> Tuple[int, int, int, int]:
    """Shape of a uint8 4-bit cache: 9/8 head_dim bytes per token and kv head hold its key and value."""
    return num_kv4_pages, num_kv_heads, page_size, 9 * head_dim // 8


def cosa_kv4_attention_workspace_size(p: CosaKvParams, with_weights: bool = False) -> int:
    """Bytes of workspace; 0 if the call would refuse ``p``."""
    return int(kv_library().cosa_kv4_attention_workspace_size(ctypes.byref(p), int(with_weights)))


def kv_required_numel(p: CosaKvParams) -> dict:
    """Elements that each buffer must hold at least (the layouts of include/cosa_kv.h)."""
    tables = p.num_reqs * p.max_pages_per_req
    cache = p.num_pages * p.page_size * p.num_kv_heads * p.head_dim
    q = p.total_tokens * p.num_q_heads * p.head_dim
    weights = p.num_reqs * p.num_kv_heads * p.max_seqlen
    return {"q_out": q, "out": q, "k_out": p.total_tokens * p.num_kv_heads * p.head_dim, "k_cache": cache,
            "v_cache": cache, "kv4_cache": p.num_kv4_pages * p.num_kv_heads * p.page_size * 9 * p.head_dim // 8,
            "page_table": tables, "src_page_table": tables, "dst_page_table": tables,
            "evict_page_table": p.num_reqs * p.max_dst_pages, "cu_seqlens": p.num_reqs + 1, "start": p.num_reqs,
            "kv_len": p.num_reqs, "new_len": p.num_reqs, "positions": p.total_tokens, "inv_freq": p.rotary_dim // 2,
            "q_weight": p.head_dim, "k_weight": p.head_dim, "weights": weights, "weights_out": weights,
            "kept": p.num_reqs * p.num_kv_heads * p.budget, "status": 1}


@functools.lru_cache(maxsize=256)
def _sizes(params: bytes) -> dict:
    """kv_required_numel by the parameters' values."""
    return kv_required_numel(CosaKvParams.from_buffer_copy(params))


class _Call:
    """Checks of one call's tensors and its stream.  The first tensor sets the device."""

    __slots__ = ("p", "need", "index")

    def __init__(self, p: CosaKvParams):
        self.p, self.need, self.index = p, _sizes(bytes(p)), None

    def on_device(self, t: torch.Tensor, name: str) -> None:
        index = t.get_device()
        if index == self.index:
            return
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if self.index is not None:
            raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{self.index}")
        self.index = index

    def dense(self, *wanted, **keys) -> list:
        """Addresses of contiguous tensors (tensor or None, name, dtype) of at least the sizes that the parameters imply
        (`keys`: names whose size stands under another one)."""
        out, need, index = [], self.need, self.index
        if keys:
            need = {**need, **{name: need[key] for name, key in keys.items()}}
        for t, name, dtype in wanted:
            if t is None:
                out.append(None)
                continue
            if t.dtype is not dtype or not t.is_contiguous() or t.numel() < need[name] or t.get_device() != index:
                self.look(t, name, dtype, need[name])
                index = self.index
            out.append(t.data_ptr())
        return out

    def look(self, t: torch.Tensor, name: str, dtype: torch.dtype, least: int) -> None:
        """What is wrong with a tensor, unless it is the first one on a device."""
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.numel() < least:
            raise ValueError(f"{name} holds {t.numel()} elements; the parameters need at least {least}")
        self.on_device(t, name)

    def rows(self, t: torch.Tensor, name: str, heads: int):
        """Address and token stride of rows [total_tokens, heads, d], whose tokens may lie apart."""
        p = self.p
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
        shape, d = t.shape, p.head_dim
        if len(shape) != 3 or shape[1] != heads or shape[2] != d:
            raise ValueError(f"{name} must be [total_tokens, {heads}, {d}], got {list(shape)}")
        if shape[0] < p.total_tokens:
            raise ValueError(f"{name} holds {shape[0]} tokens; the parameters need at least {p.total_tokens}")
        st = t.stride()
        if shape[0] and (st[2] != 1 or (heads > 1 and st[1] != d)):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        if shape[0] > 1 and st[0] < heads * d:
            raise ValueError(f"{name}: tokens are {st[0]} elements apart, a token has {heads * d}")
        self.on_device(t, name)
        # the stride of a single token says nothing
        return t.data_ptr(), (st[0] if shape[0] > 1 else 0)

    def params(self, **strides) -> CosaKvParams:
        """The parameters with this call's strides (a copy: the caller's stay as they are)."""
        p = CosaKvParams.from_buffer_copy(self.p)
        for n, s in strides.items():
            setattr(p, n, s)
        return p

    def run(self, name: str, p: CosaKvParams, args, status: Optional[torch.Tensor], stream) -> None:
        if status is not None:
            (status,) = self.dense((status, "status", torch.int32))
        if stream is None:
            s = _current_stream(self.index)
        elif stream.device.index == self.index:
            s = stream.cuda_stream
        else:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{self.index}")
        f = getattr(_lib or kv_library(), name)
        if torch.cuda.current_device() == self.index:
            rc = f(p, *args, status, s)
        else:
            with torch.cuda.device(self.index):
                rc = f(p, *args, status, s)
        if rc != COSA_OK:
            raise CosaError(rc, name)

    def empty(self, shape, dtype: torch.dtype, stream) -> torch.Tensor:
        """Memory for an output or workspace, tied to the stream that the call runs on."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.index))
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.index))


def cosa_qk_norm_rope(p: CosaKvParams, q: torch.Tensor, k: torch.Tensor, cu_seqlens: torch.Tensor, inv_freq: torch.Tensor,
                      *, v: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                      k_weight: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                      start: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                      k_out: Optional[torch.Tensor] = None, k_cache: Optional[torch.Tensor] = None,
                      v_cache: Optional[torch.Tensor] = None, page_table: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Norm and rotation of q [T, Hq, d] and k [T, Hkv, d] (bf16; tokens may lie apart, as in the slices of a
    fused projection).  With k_cache, v_cache, page_table and v, keys and values go to the pages; else k goes
    to rows.  Returns (q_out, k_out), k_out None if it was not asked for and the pages were given."""
    c = _Call(p)
    qp, qs = c.rows(q, "q", p.num_q_heads)
    kp, ks = c.rows(k, "k", p.num_kv_heads)
    vp, vs = (None, 0) if v is None else c.rows(v, "v", p.num_kv_heads)
    if q_out is None:
        q_out = c.empty((p.total_tokens, p.num_q_heads, p.head_dim), torch.bfloat16, stream)
    if k_out is None and k_cache is None:
        k_out = c.empty((p.total_tokens, p.num_kv_heads, p.head_dim), torch.bfloat16, stream)
    bf, i32 = torch.bfloat16, torch.int32
    args = c.dense((q_weight, "q_weight", bf), (k_weight, "k_weight", bf), (inv_freq, "inv_freq", torch.float64),
                   (positions, "positions", i32), (cu_seqlens, "cu_seqlens", i32), (start, "start", i32), (q_out, "q_out", bf),
                   (k_out, "k_out", bf), (k_cache, "k_cache", bf), (v_cache, "v_cache", bf), (page_table, "page_table", i32))
    c.run("cosa_qk_norm_rope", c.params(q_stride=qs, k_stride=ks, v_stride=vs), (qp, kp, vp, *args), status, stream)
    return q_out, k_out


def cosa_kv4_store(p: CosaKvParams, kv4_cache: torch.Tensor, page_table: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                   cu_seqlens: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
                   src_page_table: Optional[torch.Tensor] = None, kv_len: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """K and V into the 4-bit cache: rows k, v [T, Hkv, d] packed by cu_seqlens, the first of request b to slot
    start[b]; or, with src_page_table and kv_len, the bf16 pages k, v, slots start[b] .. kv_len[b] - 1."""
    c = _Call(p)
    bf, i32 = torch.bfloat16, torch.int32
    if src_page_table is None:
        if cu_seqlens is None:
            raise ValueError("rows need cu_seqlens")
        kp, ks = c.rows(k, "k", p.num_kv_heads)
        vp, vs = c.rows(v, "v", p.num_kv_heads)
    else:
        if kv_len is None:
            raise ValueError("pages need kv_len")
        (kp, vp), ks, vs = c.dense((k, "k", bf), (v, "v", bf), k="k_cache", v="v_cache"), 0, 0
    args = c.dense((cu_seqlens, "cu_seqlens", i32), (src_page_table, "src_page_table", i32), (start, "start", i32),
                   (kv_len, "kv_len", i32), (kv4_cache, "kv4_cache", torch.uint8), (page_table, "page_table", i32))
    c.run("cosa_kv4_store", c.params(k_stride=ks, v_stride=vs), (kp, vp, *args), status, stream)


def cosa_kv4_load(p: CosaKvParams, kv4_cache: torch.Tensor, page_table: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, dst_page_table: torch.Tensor, *, kv_len: torch.Tensor,
                  start: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Slots start[b] .. kv_len[b] - 1 of the 4-bit cache into the bf16 pages of dst_page_table."""
    c = _Call(p)
    bf, i32 = torch.bfloat16, torch.int32
    args = c.dense((kv4_cache, "kv4_cache", torch.uint8), (page_table, "page_table", i32), (start, "start", i32),
                   (kv_len, "kv_len", i32), (k_cache, "k_cache", bf), (v_cache, "v_cache", bf),
                   (dst_page_table, "dst_page_table", i32))
    c.run("cosa_kv4_load", p, args, status, stream)


def cosa_kv4_attention(p: CosaKvParams, q: torch.Tensor, cu_seqlens: torch.Tensor, kv4_cache: torch.Tensor,
                       page_table: torch.Tensor, kv_len: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                       weights: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the newest tokens q [T, Hq, d] (request b's are the last of its kv_len[b] slots) over the 4-bit
    cache; returns out bf16 [T, Hq, d].  weights, float32 [B, Hkv, max_seqlen], is added to in place.  A workspace
    that is given must be large enough and not in use by another call; without one it is allocated here."""
    c = _Call(p)
    bf, i32 = torch.bfloat16, torch.int32
    qp, qs = c.rows(q, "q", p.num_q_heads)
    if out is None:
        out = c.empty((p.total_tokens, p.num_q_heads, p.head_dim), bf, stream)
    args = c.dense((cu_seqlens, "cu_seqlens", i32), (kv4_cache, "kv4_cache", torch.uint8), (page_table, "page_table", i32),
                   (kv_len, "kv_len", i32), (out, "out", bf), (weights, "weights", torch.float32))
    if workspace is None:
        size = cosa_kv4_attention_workspace_size(p, weights is not None)
        workspace = c.empty(max(size, 256), torch.uint8, stream)
    c.on_device(workspace, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    args += [workspace.data_ptr(), workspace.numel() * workspace.element_size()]
    c.run("cosa_kv4_attention", c.params(q_stride=qs) if qs else p, (qp, *args), status, stream)
    return out


def cosa_kv4_evict(p: CosaKvParams, kv4_cache: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                   weights: torch.Tensor, dst_page_table: torch.Tensor, *, new_len: Optional[torch.Tensor] = None,
                   kept: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Keeps p.budget slots per request and kv head and moves them, in order, to the pages of dst_page_table (pages
    of the same cache that hold none of the sources).  Returns (new_len [B], kept [B, Hkv, budget], weights_out)."""
    c = _Call(p)
    i32 = torch.int32
    (kv4,) = c.dense((kv4_cache, "kv4_cache", torch.uint8))
    if new_len is None:
        new_len = c.empty((p.num_reqs,), i32, stream)
    if kept is None:
        kept = c.empty((p.num_reqs, p.num_kv_heads, p.budget), i32, stream)
    if weights_out is None:
        weights_out = c.empty((p.num_reqs, p.num_kv_heads, p.max_seqlen), torch.float32, stream)
    args = c.dense((page_table, "page_table", i32), (kv_len, "kv_len", i32), (weights, "weights", torch.float32),
                   (dst_page_table, "dst_page_table", i32), (new_len, "new_len", i32), (kept, "kept", i32),
                   (weights_out, "weights_out", torch.float32), dst_page_table="evict_page_table")
    c.run("cosa_kv4_evict", p, (kv4, *args), status, stream)
    return new_len, kept, weights_out
