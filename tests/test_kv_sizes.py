"""Sizes that libcosa_kv states on the host, at the ends of what the parameters can hold; no GPU."""
import ctypes

import pytest

from tests.test_kv_abi import C, F, attend, params  # noqa: F401  (C: the fixture that builds and loads the library)

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5


def huge(C, total_tokens, heads, max_seqlen=1 << 30):
    return params(C, num_reqs=1, num_q_heads=heads, num_kv_heads=heads, total_tokens=total_tokens, max_seqlen=max_seqlen,
                  max_pages_per_req=1 << 24)


def test_workspace_of_more_bytes_than_64_bits_number(C):
    """The weights' logits take rows * slots * 4 bytes: what does not fit 64 bits (its remainder would be a small size, and
    the kernel would write past it) has no size and is refused."""
    for total, heads in ((1 << 29, 8), (1 << 30, 4), (1 << 30, 8), (1 << 30, 65535)):       # 2^64 bytes and more
        p = huge(C, total, heads)
        assert C.cosa_kv4_attention_workspace_size(p, with_weights=True) == 0, (total, heads)
        assert attend(C, p, w=F) == UNSUPPORTED
        assert C.cosa_kv4_attention_workspace_size(p) > 0                                   # without weights no such memory
        assert attend(C, p, size=1) == WORKSPACE
    total, heads = 1 << 26, 4                                                               # 2^60 bytes
    size = C.cosa_kv4_attention_workspace_size(huge(C, total, heads), with_weights=True)
    assert size > total * heads * (1 << 30) * 4
    assert attend(C, huge(C, total, heads), w=F, size=1 << 40) == WORKSPACE


def test_no_workspace_for_parameters_that_the_attention_refuses(C):
    assert C.cosa_kv4_attention_workspace_size(params(C)) > 0
    for kw in (dict(max_new_tokens=0), dict(num_kv4_pages=0), dict(sm_scale=0.0), dict(sm_scale=float("nan")), dict(sm_scale=1e30),
               dict(q_stride=2048), dict(total_tokens=-1), dict(max_seqlen=0), dict(max_pages_per_req=15), dict(num_q_heads=7),
               dict(total_tokens=1 << 30, num_q_heads=8, num_kv_heads=1), dict(flags=2)):
        p = params(C, **kw)
        assert attend(C, p) in (INVALID, UNSUPPORTED), kw
        for weights in (False, True):
            assert C.cosa_kv4_attention_workspace_size(p, with_weights=weights) == 0, kw
