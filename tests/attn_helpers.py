"""Inputs shared by the tests of include/cosa_attn.h's calls."""
from __future__ import annotations

import numpy as np
import torch

from block_sparse_long_gb300 import attn as C
from tests import attn_reference as ref
from tests.kv_helpers import bf, cu_of, i32, table
from tests.kv_reference import bf16, to_f64

DEV = "cuda"
LN2 = 0.6931471805599453


def random_masks(rng, new, ragged=False):
    """Masks of a random tree: the node and those above it; ragged: any bits, some rows without their own."""
    masks = []
    for i in range(new):
        if ragged:
            masks.append(int(rng.integers(0, 1 << min(new, 62))) if i % 3 else 0)
        else:
            up = int(rng.integers(-1, i)) if i else -1
            masks.append((masks[up] if up >= 0 else 0) | 1 << i)
    return masks


def bits(masks):
    """int64 tensor of all requests' masks."""
    flat = [m - (1 << 64) if m >> 63 else m for req in masks for m in req]
    return torch.tensor(flat, dtype=torch.int64, device=DEV)


def garbage(rng, *shape):
    """bf16 memory full of NaN, infinities and large values."""
    x = torch.from_numpy(rng.choice(np.array([np.nan, np.inf, -np.inf, 3e38, -1.0], np.float32), size=shape))
    return x.to(torch.bfloat16).to(DEV)


def pages_of(rng, rows, t, total, P):
    """Caches of garbage with rows[b] [len, ...] (bf16 values) in the slots that have a page."""
    cache = garbage(rng, total, P, *rows[0].shape[1:])
    host = cache.cpu()
    for b, x in enumerate(rows):
        x = torch.from_numpy(x).to(torch.bfloat16)
        for at in range(0, x.shape[0], P):
            phys = int(t[b, at // P])
            if 0 <= phys < total:
                host[phys, :min(P, x.shape[0] - at)] = x[at:at + P]
    return host.to(DEV)


def there_of(t, b, n, P, total):
    e = t[b].astype(np.int64)
    ok = (e >= 0) & (e < total)
    return ok[np.arange(n) // P]


class Paged:
    """A batch for one of the attentions over pages, in garbage, with its reference."""

    def __init__(self, seed, lens, new, Hq, Hkv=1, d=128, P=64, latent=0, tree=False, ragged=False, missing=(), spare=3, strided=False,
                 scale=None, edit=None, pitch=None):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.new, self.P, self.latent = lens, new, P, latent
        B, T = len(lens), sum(new)
        pages = pitch or max(1, max(-(-n // P) for n in lens))
        total = B * pages + 2
        self.t = table(rng, B, pages, total, missing)
        dk = latent + 64 if latent else d
        heads = 1 if latent else Hkv
        ks = [bf16(rng.standard_normal((n, heads, dk))) for n in lens]
        vs = [k[..., :latent] for k in ks] if latent else [bf16(rng.standard_normal((n, heads, d)) * 0.8) for n in lens]
        q = bf16(rng.standard_normal((T, Hq, dk)) * 1.3)
        if edit is not None:
            edit(ks, vs, q)
        self.masks = [random_masks(rng, n, ragged) for n in new] if tree else None
        self.scale = scale or ((dk if latent == 0 else 192) ** -0.5)
        self.p = C.make_attn_params(num_reqs=B, num_q_heads=Hq, num_kv_heads=heads, head_dim=d, latent_dim=latent or 512, page_size=P,
                                    total_tokens=T + spare, max_seqlen=pages * P, num_pages=total, max_pages_per_req=pages,
                                    max_new_tokens=max(1, max(new)), sm_scale=self.scale)
        if latent:
            self.cache = pages_of(rng, [k[:, 0] for k in ks], self.t, total, P)
        else:
            self.k, self.v = pages_of(rng, ks, self.t, total, P), pages_of(rng, vs, self.t, total, P)

        def rows(x):
            y = torch.from_numpy(np.concatenate([x, np.ones((spare, *x.shape[1:]))])).to(torch.bfloat16).to(DEV)
            if strided == "heads":      # head by head, as a batched product leaves them
                y = y.transpose(0, 1).contiguous().transpose(0, 1)
            elif strided:     # tokens apart, as in the slice of a fused projection
                wide = torch.zeros(y.shape[0], y[0].numel() + 48, dtype=torch.bfloat16, device=DEV)
                wide[:, 16:16 + y[0].numel()] = y.flatten(1)
                y = wide[:, 16:16 + y[0].numel()].unflatten(1, y.shape[1:])
            return y

        self.q, self.q_rope = (rows(q[..., :latent]), rows(q[..., latent:])) if latent else (rows(q), None)
        self.cu, self.kv_len, self.pt = cu_of(new), i32(lens), i32(self.t)
        self.mask = None if self.masks is None else torch.cat([bits(self.masks), torch.full((spare,), -1, dtype=torch.int64, device=DEV)])
        self.T, self.spare, self.Hq, self.dv = T, spare, Hq, latent or d
        self.ks, self.vs, self.qf, self.total = ks, vs, q, total

    def buffers(self):
        """out and lse full of noise."""
        out = bf(self.rng, self.T + self.spare, self.Hq, self.dv)
        return out, torch.randn(self.T + self.spare, self.Hq, device=DEV)

    def call(self, **kw):
        kw.setdefault("tree_mask", self.mask)
        if self.latent:
            return C.cosa_latent_attention(kw.pop("p", self.p), self.q, self.q_rope, self.cu, self.cache, self.pt, self.kv_len, **kw)
        return C.cosa_tree_attention(kw.pop("p", self.p), self.q, self.cu, self.k, self.v, self.pt, self.kv_len, **kw)

    def check(self, out, lse, skip=()):
        """out and lse [tokens, ...] against the reference; rows of the requests in `skip` are not looked at."""
        got, got_lse = to_f64(out), None if lse is None else to_f64(lse)
        row = 0
        for b, n in enumerate(self.new):
            if b not in skip:
                L = self.lens[b]
                seen = ref.seen_of(L, n, None if self.masks is None else self.masks[b]) & there_of(self.t, b, L, self.P, self.total)
                want = ref.attention(self.qf[row:row + n], self.ks[b], self.vs[b], seen, self.scale)
                near(got[row:row + n], None if lse is None else got_lse[row:row + n], *want, L)
            row += n


def near(out, lse, want, want_lse, mag, err, L):
    """Outputs: half a bf16 step of the result, and of each p (its rounding for the second product), 2.1 times the logits'
    error, and for the fp32 sum that truncates 2^-23 at each of L / 16 steps, the joins of the parts and the exponential 2^-18 and that.
    lse: the logits' error, the sum's (L + 64 additions of 2^-24 and 2^-22 of the exponential) and its own rounding."""
    assert np.array_equal(np.isnan(out), np.isnan(want)), "NaN"
    fine = np.isfinite(want)
    assert np.array_equal(out[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    slack = np.abs(want) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.1 * err[..., None] + L * 2.0 ** -27 + 2.0 ** -18)
    off = np.abs(out - want)[fine] - slack[fine]
    assert not off.size or off.max() <= 1e-30, float(off.max())
    if lse is None:
        return
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), none) and np.array_equal(np.isnan(lse), np.isnan(want_lse))
    fine = np.isfinite(want_lse)
    slack = err + (L + 64) * 2.0 ** -24 + 2.0 ** -21 + np.abs(np.where(fine, want_lse, 0.0)) * 2.0 ** -22
    off = np.abs(lse[fine] - want_lse[fine]) - slack[fine]
    assert not off.size or off.max() <= 0, float(off.max())
