"""Thin Python binding of libcosa_attn's C ABI (include/cosa_attn.h): dense attention beside the sparse prefill, for trees of
drafted tokens and for latent attention.

Argument marshalling only, as in :mod:`block_sparse_long_gb300.kv`: every step runs in the CUDA kernels of libcosa_attn.so,
PyTorch supplies device memory and streams, and there is no fallback.

The functions carry the C names:
  cosa_tree_attention     attention of the newest tokens, drafted trees among them, over the prefill's bf16 pages
  cosa_tree_commit        the accepted path of each tree moved behind its context
  cosa_latent_rope        latent attention's norm and rotation, and the cache write
  cosa_latent_attention   attention of the newest tokens over pages of latent vectors (absorbed form)
  cosa_latent_prefill     causal attention of prompts with keys and values expanded per head
  cosa_tree_attention_workspace_size, cosa_latent_attention_workspace_size, cosa_attn_version

A step with drafted tokens over one layer (kv_len counts them)::

    q_out, _ = cosa_qk_norm_rope(kp, q, k, cu, inv_freq, v=v, positions=depth, start=kv_len - new, k_cache=k_cache,
                                 v_cache=v_cache, page_table=pt)                    # block_sparse_long_gb300.kv
    out = cosa_tree_attention(p, q_out, cu, k_cache, v_cache, pt, kv_len, tree_mask=mask)
    kv_len = cosa_tree_commit(p, (k_cache, v_cache), cu, pt, kv_len, path, path_len)

and of latent attention, a prompt and then new tokens::

    q_rope, c, k_rope = cosa_latent_rope(p, kv, cu, inv_freq, q=q[..., d:], weight=w, c_out=c, k_out=k_rope, cache=cache,
                                         page_table=pt)
    out = cosa_latent_prefill(p, q[..., :d], q_rope, k_nope, k_rope, v, cu)         # k_nope, v = c's products with the weights
    q_rope, _, _ = cosa_latent_rope(p1, kv, cu1, inv_freq, q=q[..., d:], weight=w, start=kv_len - new, cache=cache,
                                    page_table=pt)
    out = cosa_latent_attention(p1, q_latent, q_rope, cu1, cache, pt, kv_len)

Every call checks the tensors' types, sizes and device on the host, runs on the current stream of the tensors' device (or
``stream``), and takes an optional int32 ``status`` tensor, zeroed by the caller, that receives errors found on the device.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Sequence, Tuple

import torch

from .kv import _Call

_HERE = os.path.dirname(os.path.abspath(__file__))
ATTN_LIB_PATH = os.path.join(_HERE, "libcosa_attn.so")

# Every symbol include/cosa_attn.h declares.
ATTN_EXPORTS = ("cosa_attn_version", "cosa_tree_attention_workspace_size", "cosa_tree_attention", "cosa_tree_commit",
                "cosa_latent_rope", "cosa_latent_attention_workspace_size", "cosa_latent_attention", "cosa_latent_prefill")
COSA_ATTN_ROPE_DIM = 64
COSA_ATTN_MAX_TREE = 64
COSA_ATTN_FLAG_INTERLEAVED = 1
COSA_ATTN_FLAG_TEST_STALL = 4   # test hook of the attentions: every in-kernel wait runs out


class CosaAttnParams(ctypes.Structure):
    """Mirror of ``cosa_attn_params``."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_reqs", "num_q_heads", "num_kv_heads", "head_dim", "latent_dim", "page_size", "total_tokens", "total_kv_tokens",
        "max_seqlen", "num_pages", "max_pages_per_req", "max_new_tokens", "flags", "reserved")] + [(n, ctypes.c_int64) for n in (
            "q_stride", "q_head_stride", "q_rope_stride", "q_rope_head_stride", "k_stride", "k_head_stride", "k_rope_stride",
            "v_stride", "v_head_stride")] + [("sm_scale", ctypes.c_double), ("norm_eps", ctypes.c_double)]


_lib = None


def attn_library() -> ctypes.CDLL:
    """Load libcosa_attn.so once.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(ATTN_LIB_PATH):
        raise RuntimeError(f"{ATTN_LIB_PATH} is missing: build it with `python -m block_sparse_long_gb300.build`")
    lib = ctypes.CDLL(ATTN_LIB_PATH)
    vp, sz, pp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(CosaAttnParams)
    lib.cosa_attn_version.restype = ctypes.c_int
    for name, args in (("cosa_tree_attention", [vp] * 10 + [sz, vp, vp]), ("cosa_latent_attention", [vp] * 10 + [sz, vp, vp]),
                       ("cosa_tree_commit", [vp, vp, ctypes.c_int32] + [vp] * 8), ("cosa_latent_rope", [vp] * 14),
                       ("cosa_latent_prefill", [vp] * 11)):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [pp] + args
        if name.endswith("_attention"):
            f = getattr(lib, name + "_workspace_size")
            f.restype, f.argtypes = sz, [pp]
    _lib = lib
    return lib


def cosa_attn_version() -> int:
    return int(attn_library().cosa_attn_version())


def make_attn_params(*, num_reqs, num_q_heads, num_kv_heads=1, head_dim=128, latent_dim=512, page_size=64, total_tokens=0,
                     total_kv_tokens=0, max_seqlen=1, num_pages=1, max_pages_per_req=1, max_new_tokens=1, interleaved=False,
                     sm_scale=None, norm_eps=1e-6) -> CosaAttnParams:
    """sm_scale defaults to 1/sqrt(head_dim), the tree attention's; latent attention's is 1/sqrt(head_dim + 64)."""
    return CosaAttnParams(
        num_reqs=num_reqs, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim, latent_dim=latent_dim,
        page_size=page_size, total_tokens=total_tokens, total_kv_tokens=total_kv_tokens, max_seqlen=max_seqlen,
        num_pages=num_pages, max_pages_per_req=max_pages_per_req, max_new_tokens=max_new_tokens,
        flags=COSA_ATTN_FLAG_INTERLEAVED if interleaved else 0,
        sm_scale=float(sm_scale if sm_scale is not None else 1.0 / math.sqrt(head_dim)), norm_eps=float(norm_eps))


def latent_cache_shape(num_pages: int, page_size: int, latent_dim: int) -> Tuple[int, int, int]:
    """Shape of a bf16 cache of latent vectors."""
    return num_pages, page_size, latent_dim + COSA_ATTN_ROPE_DIM


def cosa_tree_attention_workspace_size(p: CosaAttnParams) -> int:
    """Bytes of workspace; 0 if the call would refuse ``p``."""
    return int(attn_library().cosa_tree_attention_workspace_size(ctypes.byref(p)))


def cosa_latent_attention_workspace_size(p: CosaAttnParams) -> int:
    """Bytes of workspace; 0 if the call would refuse ``p``."""
    return int(attn_library().cosa_latent_attention_workspace_size(ctypes.byref(p)))


def attn_required_numel(p: CosaAttnParams) -> dict:
    """Elements that each buffer must hold at least (the layouts of include/cosa_attn.h)."""
    slots, rows, rope = p.num_pages * p.page_size, p.total_tokens * p.num_q_heads, COSA_ATTN_ROPE_DIM
    cache = slots * p.num_kv_heads * p.head_dim
    return {"out": rows * p.head_dim, "latent_out": rows * p.latent_dim, "lse": rows, "q_out": rows * rope,
            "c_out": p.total_tokens * p.latent_dim, "k_out": p.total_tokens * rope, "k_cache": cache, "v_cache": cache,
            "latent_cache": slots * (p.latent_dim + rope), "page_table": p.num_reqs * p.max_pages_per_req,
            "cu_seqlens": p.num_reqs + 1, "cu_kv": p.num_reqs + 1, "start": p.num_reqs, "kv_len": p.num_reqs,
            "new_len": p.num_reqs, "path_len": p.num_reqs, "path": p.num_reqs * p.max_new_tokens,
            "tree_mask": p.total_tokens, "positions": p.total_tokens, "inv_freq": rope // 2, "weight": p.latent_dim, "status": 1}


@functools.lru_cache(maxsize=256)
def _sizes(params: bytes) -> dict:
    """attn_required_numel by the parameters' values."""
    return attn_required_numel(CosaAttnParams.from_buffer_copy(params))


class _AttnCall(_Call):
    """The checks of a call of this library."""

    __slots__ = ()

    def __init__(self, p: CosaAttnParams):
        self.p, self.need, self.index = p, _sizes(bytes(p)), None

    def strided(self, t: torch.Tensor, name: str, tokens: int, heads: Optional[int], width: int):
        """Address, token stride and head stride of rows [tokens, heads, width] (heads None: [tokens, width]), whose tokens
        and heads may lie apart."""
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
        want = (width,) if heads is None else (heads, width)
        if t.dim() != 1 + len(want) or tuple(t.shape[1:]) != want:
            raise ValueError(f"{name} must be [tokens, {', '.join(map(str, want))}], got {list(t.shape)}")
        if t.shape[0] < tokens:
            raise ValueError(f"{name} holds {t.shape[0]} tokens; the parameters need at least {tokens}")
        st, heads = t.stride(), heads or 1
        # the stride of a single token or head says nothing
        by_head = st[1] if len(want) == 2 and heads > 1 else width
        by_token = st[0] if t.shape[0] > 1 else max(heads * width, (heads - 1) * by_head + width)
        if t.shape[0]:
            if st[-1] != 1:
                raise ValueError(f"{name}: the values of a head must be contiguous")
            if by_head < width:
                raise ValueError(f"{name}: heads are {by_head} elements apart, a head has {width}")
            if t.shape[0] > 1 and by_token < (heads - 1) * by_head + width:
                raise ValueError(f"{name}: tokens are {by_token} elements apart, a token has {(heads - 1) * by_head + width}")
        self.on_device(t, name)
        if t.shape[0] <= 1:
            by_token += -by_token % 8
        return t.data_ptr(), by_token, by_head

    def params(self, **strides) -> CosaAttnParams:
        """The parameters with this call's strides (a copy: the caller's stay as they are)."""
        p = CosaAttnParams.from_buffer_copy(self.p)
        for n, s in strides.items():
            setattr(p, n, s)
        return p

    def run(self, name: str, p: CosaAttnParams, args, status, stream) -> None:
        super().run(name, p, args, status, stream, _lib or attn_library())

    def scratch(self, workspace: Optional[torch.Tensor], size_of, stream) -> list:
        """Address and bytes of the workspace, allocated here if there is none."""
        if workspace is None:
            workspace = self.empty(max(size_of(self.p), 256), torch.uint8, stream)
        self.on_device(workspace, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return [workspace.data_ptr(), workspace.numel() * workspace.element_size()]


_BF, _I32 = torch.bfloat16, torch.int32


def cosa_tree_attention(p: CosaAttnParams, q: torch.Tensor, cu_seqlens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        page_table: torch.Tensor, kv_len: torch.Tensor, *, tree_mask: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the newest tokens q [T, Hq, d] (request b's are the last of its kv_len[b] slots) over the bf16 pages;
    returns out bf16 [T, Hq, d].  Bit j of tree_mask[t] (int64): token t sees its request's token j; without it a token sees
    those up to itself.  lse, float32 [T, Hq], is written if given.  A workspace that is given must be large enough and not
    in use by another call; without one it is allocated here."""
    c = _AttnCall(p)
    qp, qs, qh = c.strided(q, "q", p.total_tokens, p.num_q_heads, p.head_dim)
    if qh != p.head_dim:
        raise ValueError("q: the heads of a token must be contiguous")
    if out is None:
        out = c.empty((p.total_tokens, p.num_q_heads, p.head_dim), _BF, stream)
    args = c.dense((cu_seqlens, "cu_seqlens", _I32), (k_cache, "k_cache", _BF), (v_cache, "v_cache", _BF),
                   (page_table, "page_table", _I32), (kv_len, "kv_len", _I32), (tree_mask, "tree_mask", torch.int64),
                   (out, "out", _BF), (lse, "lse", torch.float32))
    args += c.scratch(workspace, cosa_tree_attention_workspace_size, stream)
    c.run("cosa_tree_attention", c.params(q_stride=qs), (qp, *args), status, stream)
    return out


def cosa_tree_commit(p: CosaAttnParams, caches: Sequence[torch.Tensor], cu_seqlens: torch.Tensor, page_table: torch.Tensor,
                     kv_len: torch.Tensor, path: torch.Tensor, path_len: torch.Tensor, *, new_len: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Moves the rows of tokens path[b, 0] < path[b, 1] < ... (path_len[b] of them) of each request's tree to the slots behind
    its context, in the one or two caches given ([pages, P, Hkv, d] keys and values, or [pages, P, latent_dim + 64]); returns
    new_len [B], the requests' lengths after it."""
    c = _AttnCall(p)
    caches = tuple(caches)
    if len(caches) not in (1, 2) or any(x.dtype != _BF or x.dim() < 3 or not x.is_contiguous() for x in caches):
        raise ValueError("caches: one or two contiguous bf16 tensors [num_pages, page_size, ...]")
    row = math.prod(caches[0].shape[2:])
    for x in caches:
        if x.shape[0] < p.num_pages or x.shape[1] != p.page_size or math.prod(x.shape[2:]) != row:
            raise ValueError(f"caches must be [{p.num_pages}, {p.page_size}, ...] with equal rows, got {list(x.shape)}")
    for x in caches:
        c.on_device(x, "caches")
    if new_len is None:
        new_len = c.empty((p.num_reqs,), _I32, stream)
    args = c.dense((cu_seqlens, "cu_seqlens", _I32), (page_table, "page_table", _I32), (kv_len, "kv_len", _I32), (path, "path", _I32),
                   (path_len, "path_len", _I32), (new_len, "new_len", _I32))
    second = caches[1].data_ptr() if len(caches) == 2 else None
    c.run("cosa_tree_commit", p, (caches[0].data_ptr(), second, row, *args), status, stream)
    return new_len


def cosa_latent_rope(p: CosaAttnParams, kv: torch.Tensor, cu_seqlens: torch.Tensor, inv_freq: torch.Tensor, *,
                     q: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None, c_out: Optional[torch.Tensor] = None,
                     k_out: Optional[torch.Tensor] = None, cache: Optional[torch.Tensor] = None,
                     page_table: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None):
    """Norm of the latent part and rotation of the rest of kv [T, latent_dim + 64], and rotation of q [T, Hq, 64] (tokens and
    heads may lie apart, as in a slice of the query projection).  With cache and page_table they go to the pages, with c_out
    [T, latent_dim] and k_out [T, 64], or without either, to rows.  Returns (q_out, c_out, k_out), None where there is none."""
    c = _AttnCall(p)
    rope = COSA_ATTN_ROPE_DIM
    kvp, kvs, _ = c.strided(kv, "kv", p.total_tokens, None, p.latent_dim + rope)
    qp, qs, qh = (None, 0, 0) if q is None else c.strided(q, "q", p.total_tokens, p.num_q_heads, rope)
    if q is not None and q_out is None:
        q_out = c.empty((p.total_tokens, p.num_q_heads, rope), _BF, stream)
    if c_out is None and k_out is None and cache is None:
        c_out = c.empty((p.total_tokens, p.latent_dim), _BF, stream)
        k_out = c.empty((p.total_tokens, rope), _BF, stream)
    args = c.dense((weight, "weight", _BF), (inv_freq, "inv_freq", torch.float64), (positions, "positions", _I32),
                   (cu_seqlens, "cu_seqlens", _I32), (start, "start", _I32), (q_out, "q_out", _BF), (c_out, "c_out", _BF),
                   (k_out, "k_out", _BF), (cache, "latent_cache", _BF), (page_table, "page_table", _I32))
    c.run("cosa_latent_rope", c.params(k_stride=kvs, q_rope_stride=qs, q_rope_head_stride=qh), (kvp, qp, *args), status, stream)
    return q_out, c_out, k_out


def cosa_latent_attention(p: CosaAttnParams, q_latent: torch.Tensor, q_rope: torch.Tensor, cu_seqlens: torch.Tensor,
                          cache: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, *,
                          tree_mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the newest tokens, queries q_latent [T, Hq, latent_dim] and q_rope [T, Hq, 64], over the pages of latent
    vectors; returns out bf16 [T, Hq, latent_dim].  The rest as in cosa_tree_attention."""
    c = _AttnCall(p)
    qp, qs, qh = c.strided(q_latent, "q_latent", p.total_tokens, p.num_q_heads, p.latent_dim)
    rp, rs, rh = c.strided(q_rope, "q_rope", p.total_tokens, p.num_q_heads, COSA_ATTN_ROPE_DIM)
    if qh != p.latent_dim or rh != COSA_ATTN_ROPE_DIM:
        raise ValueError("q_latent, q_rope: the heads of a token must be contiguous")
    if out is None:
        out = c.empty((p.total_tokens, p.num_q_heads, p.latent_dim), _BF, stream)
    args = c.dense((cu_seqlens, "cu_seqlens", _I32), (cache, "latent_cache", _BF), (page_table, "page_table", _I32),
                   (kv_len, "kv_len", _I32), (tree_mask, "tree_mask", torch.int64), (out, "out", _BF), (lse, "lse", torch.float32),
                   out="latent_out")
    args += c.scratch(workspace, cosa_latent_attention_workspace_size, stream)
    c.run("cosa_latent_attention", c.params(q_stride=qs, q_rope_stride=rs), (qp, rp, *args), status, stream)
    return out


def cosa_latent_prefill(p: CosaAttnParams, q_nope: torch.Tensor, q_rope: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor,
                        v: torch.Tensor, cu_seqlens: torch.Tensor, *, cu_kv: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Causal attention of prompts packed by cu_seqlens: queries q_nope [T, Hq, d] and q_rope [T, Hq, 64], keys k_nope
    [Tk, Hq, d] and, shared by the heads, k_rope [Tk, 64], values v [Tk, Hq, d], packed by cu_kv (without it, by cu_seqlens; a
    request's queries are the last of its keys); tokens and heads may lie apart.  Returns out bf16 [T, Hq, d]."""
    c = _AttnCall(p)
    H, d, rope, T, Tk = p.num_q_heads, p.head_dim, COSA_ATTN_ROPE_DIM, p.total_tokens, p.total_kv_tokens
    qp, qs, qh = c.strided(q_nope, "q_nope", T, H, d)
    rp, rs, rh = c.strided(q_rope, "q_rope", T, H, rope)
    kp, ks, kh = c.strided(k_nope, "k_nope", Tk, H, d)
    krp, krs, _ = c.strided(k_rope, "k_rope", Tk, None, rope)
    vp, vs, vh = c.strided(v, "v", Tk, H, d)
    if out is None:
        out = c.empty((T, H, d), _BF, stream)
    args = c.dense((cu_seqlens, "cu_seqlens", _I32), (cu_kv, "cu_kv", _I32), (out, "out", _BF), (lse, "lse", torch.float32))
    strides = dict(q_stride=qs, q_head_stride=qh, q_rope_stride=rs, q_rope_head_stride=rh, k_stride=ks, k_head_stride=kh,
                   k_rope_stride=krs, v_stride=vs, v_head_stride=vh)
    c.run("cosa_latent_prefill", c.params(**strides), (qp, rp, kp, krp, vp, *args), status, stream)
    return out
