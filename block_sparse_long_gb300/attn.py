"""Thin Python binding of libcosa_attn's C ABI (include/cosa_attn.h): dense attention beside the sparse prefill, for trees of
drafted tokens and for latent attention.

Argument marshalling only, as in :mod:`block_sparse_long_gb300.kv`: every step runs in the CUDA kernels of libcosa_attn.so,
PyTorch supplies device memory and streams, and there is no fallback.  The checks of a call's tensors and the call itself are
in the module _attn_call (csrc/attn_binding.cpp), which takes a third of the time that they take in Python.

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
import importlib
import math
import os
from typing import Optional, Sequence, Tuple

import torch

from .cosa import CosaError

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
    """Mirror of ``cosa_attn_params``.  scale_given is False, in copies too, while sm_scale is the default of make_attn_params."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_reqs", "num_q_heads", "num_kv_heads", "head_dim", "latent_dim", "page_size", "total_tokens", "total_kv_tokens",
        "max_seqlen", "num_pages", "max_pages_per_req", "max_new_tokens", "flags", "reserved")] + [(n, ctypes.c_int64) for n in (
            "q_stride", "q_head_stride", "q_rope_stride", "q_rope_head_stride", "k_stride", "k_head_stride", "k_rope_stride",
            "v_stride", "v_head_stride")] + [("sm_scale", ctypes.c_double), ("norm_eps", ctypes.c_double)]
    scale_given = True

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name == "sm_scale":
            super().__setattr__("scale_given", True)

    @classmethod
    def from_buffer_copy(cls, source, offset=0):
        made = type(cls).from_buffer_copy(cls, source, offset)
        made.scale_given = getattr(source, "scale_given", True)
        return made


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


_module = None


def _calls():
    """The module of checked calls, with the library's functions."""
    global _module
    if _module is None:
        try:
            module = importlib.import_module("._attn_call", __package__)
        except ImportError as e:
            raise RuntimeError(f"_attn_call cannot be loaded ({e}): build it with `python -m block_sparse_long_gb300.build`") from e
        lib = attn_library()
        module.bind(*(ctypes.cast(getattr(lib, "cosa_" + name), ctypes.c_void_p).value for name in (
            "tree_attention", "latent_attention", "tree_commit", "latent_rope", "latent_prefill")))
        _module = module
    return _module


def cosa_attn_version() -> int:
    return int(attn_library().cosa_attn_version())


def make_attn_params(*, num_reqs, num_q_heads, num_kv_heads=1, head_dim=128, latent_dim=512, page_size=64, total_tokens=0,
                     total_kv_tokens=0, max_seqlen=1, num_pages=1, max_pages_per_req=1, max_new_tokens=1, interleaved=False,
                     sm_scale=None, norm_eps=1e-6) -> CosaAttnParams:
    """sm_scale defaults to 1/sqrt(head_dim), the tree attention's.  Both forms of latent attention, whose scale is as a rule
    1/sqrt(d + 64) with heads of d + 64 values, refuse that default."""
    p = CosaAttnParams(
        num_reqs=num_reqs, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim, latent_dim=latent_dim,
        page_size=page_size, total_tokens=total_tokens, total_kv_tokens=total_kv_tokens, max_seqlen=max_seqlen,
        num_pages=num_pages, max_pages_per_req=max_pages_per_req, max_new_tokens=max_new_tokens,
        flags=COSA_ATTN_FLAG_INTERLEAVED if interleaved else 0,
        sm_scale=float(sm_scale if sm_scale is not None else 1.0 / math.sqrt(head_dim)), norm_eps=float(norm_eps))
    p.scale_given = sm_scale is not None
    return p


def _latent_scale(p: CosaAttnParams) -> None:
    if not p.scale_given:
        raise ValueError("sm_scale is the default of make_attn_params, the tree attention's: give latent attention its own")


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


def _empty(like: torch.Tensor, shape, dtype: torch.dtype, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """Memory for an output or workspace, tied to the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def cosa_tree_attention(p: CosaAttnParams, q: torch.Tensor, cu_seqlens: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        page_table: torch.Tensor, kv_len: torch.Tensor, *, tree_mask: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the newest tokens q [T, Hq, d] (tokens and heads may lie apart; request b's are the last of its kv_len[b]
    slots) over the bf16 pages; returns out bf16 [T, Hq, d].  Bit j of tree_mask[t] (int64): token t sees its request's token j; without it a token sees
    those up to itself.  lse, float32 [T, Hq], is written if given.  A workspace that is given must be large enough and not
    in use by another call; without one it is allocated here."""
    if out is None:
        out = _empty(q, (p.total_tokens, p.num_q_heads, p.head_dim), torch.bfloat16, stream)
    if workspace is None:
        workspace = _empty(q, max(cosa_tree_attention_workspace_size(p), 256), torch.uint8, stream)
    rc = (_module or _calls()).tree_attention(p, q, cu_seqlens, k_cache, v_cache, page_table, kv_len, tree_mask, out, lse, workspace, status, stream)
    if rc:
        raise CosaError(rc, "cosa_tree_attention")
    return out


def cosa_tree_commit(p: CosaAttnParams, caches: Sequence[torch.Tensor], cu_seqlens: torch.Tensor, page_table: torch.Tensor,
                     kv_len: torch.Tensor, path: torch.Tensor, path_len: torch.Tensor, *, new_len: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Moves the rows of tokens path[b, 0] < path[b, 1] < ... (path_len[b] of them) of each request's tree to the slots behind
    its context, in the one or two caches given ([pages, P, Hkv, d] keys and values, or [pages, P, latent_dim + 64]); returns
    new_len [B], the requests' lengths after it."""
    if len(caches) not in (1, 2):
        raise ValueError("caches: one or two contiguous bf16 tensors [num_pages, page_size, ...]")
    if new_len is None:
        new_len = _empty(caches[0], (p.num_reqs,), torch.int32, stream)
    rc = (_module or _calls()).tree_commit(p, caches[0], caches[1] if len(caches) == 2 else None, cu_seqlens, page_table, kv_len, path, path_len,
                                           new_len, status, stream)
    if rc:
        raise CosaError(rc, "cosa_tree_commit")
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
    if q is not None and q_out is None:
        q_out = _empty(kv, (p.total_tokens, p.num_q_heads, COSA_ATTN_ROPE_DIM), torch.bfloat16, stream)
    if c_out is None and k_out is None and cache is None:
        c_out = _empty(kv, (p.total_tokens, p.latent_dim), torch.bfloat16, stream)
        k_out = _empty(kv, (p.total_tokens, COSA_ATTN_ROPE_DIM), torch.bfloat16, stream)
    rc = (_module or _calls()).latent_rope(p, kv, q, weight, inv_freq, positions, cu_seqlens, start, q_out, c_out, k_out, cache, page_table,
                                           status, stream)
    if rc:
        raise CosaError(rc, "cosa_latent_rope")
    return q_out, c_out, k_out


def cosa_latent_attention(p: CosaAttnParams, q_latent: torch.Tensor, q_rope: torch.Tensor, cu_seqlens: torch.Tensor,
                          cache: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, *,
                          tree_mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of the newest tokens, queries q_latent [T, Hq, latent_dim] and q_rope [T, Hq, 64], over the pages of latent
    vectors; returns out bf16 [T, Hq, latent_dim].  p has an sm_scale of its own.  The rest as in cosa_tree_attention."""
    _latent_scale(p)
    if out is None:
        out = _empty(q_latent, (p.total_tokens, p.num_q_heads, p.latent_dim), torch.bfloat16, stream)
    if workspace is None:
        workspace = _empty(q_latent, max(cosa_latent_attention_workspace_size(p), 256), torch.uint8, stream)
    rc = (_module or _calls()).latent_attention(p, q_latent, q_rope, cu_seqlens, cache, page_table, kv_len, tree_mask, out, lse, workspace, status,
                                                stream)
    if rc:
        raise CosaError(rc, "cosa_latent_attention")
    return out


def cosa_latent_prefill(p: CosaAttnParams, q_nope: torch.Tensor, q_rope: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor,
                        v: torch.Tensor, cu_seqlens: torch.Tensor, *, cu_kv: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Causal attention of prompts packed by cu_seqlens: queries q_nope [T, Hq, d] and q_rope [T, Hq, 64], keys k_nope
    [Tk, Hq, d] and, shared by the heads, k_rope [Tk, 64], values v [Tk, Hq, d], packed by cu_kv (without it, by cu_seqlens; a
    request's queries are the last of its keys); tokens and heads may lie apart.  p has an sm_scale of its own.  Returns out bf16
    [T, Hq, d]."""
    _latent_scale(p)
    if out is None:
        out = _empty(q_nope, (p.total_tokens, p.num_q_heads, p.head_dim), torch.bfloat16, stream)
    rc = (_module or _calls()).latent_prefill(p, q_nope, q_rope, k_nope, k_rope, v, cu_seqlens, cu_kv, out, lse, status, stream)
    if rc:
        raise CosaError(rc, "cosa_latent_prefill")
    return out
