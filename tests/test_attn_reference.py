"""The tests' float64 reference of include/cosa_attn.h, against torch and small cases by hand."""
import numpy as np
import torch

from tests import attn_reference as ref


def test_attention_against_torch():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 4, 16)), rng.standard_normal((9, 2, 16)), rng.standard_normal((9, 2, 8))
    seen = ref.seen_of(9, 3, [1, 3, 4])
    assert seen[:, :6].all() and seen[:, 6:].tolist() == [[True, False, False], [True, True, False], [False, False, True]]
    out, lse, mag, err = ref.attention(q, k, v, seen, 0.3)
    kk, vv = (torch.from_numpy(x).repeat_interleave(2, 1) for x in (k, v))
    x = (torch.einsum("nhd,lhd->nhl", torch.from_numpy(q), kk) * 0.3).masked_fill(~torch.from_numpy(seen)[:, None], -np.inf)
    assert np.allclose(out, torch.einsum("nhl,lhd->nhd", x.softmax(-1), vv).numpy(), atol=1e-13)
    assert np.allclose(lse, x.logsumexp(-1).numpy(), atol=1e-13)
    assert (mag >= np.abs(out) - 1e-13).all() and (err > 0).all()


def test_nothing_seen():
    out, lse, _, _ = ref.attention(np.ones((1, 1, 4)), np.ones((2, 1, 4)), np.ones((2, 1, 4)), np.zeros((1, 2), bool), 1.0)
    assert not out.any() and np.isneginf(lse).all()


def test_chain_and_rotation_and_commit():
    assert ref.seen_of(4, 2).tolist() == [[True, True, True, False], [True] * 4]
    x = np.zeros((1, 1, 4))
    x[..., 0] = 1.0
    for inter, other in ((False, 2), (True, 1)):
        y, _ = ref.rotate(x, np.array([1]), np.array([np.pi / 2, 0.1]), inter)
        want = np.zeros(4)
        want[other] = 1.0
        assert np.allclose(y[0, 0], want)
    rows = np.arange(6.0)
    assert ref.commit(rows, np.ones(6, bool), 6, 4, [1, 3]).tolist() == [0, 1, 3, 5, 4, 5]
    assert ref.commit(rows, np.array([1, 1, 1, 1, 1, 0], bool), 6, 4, [1, 3]).tolist() == [0, 1, 3, 3, 4, 5]
    assert ref.commit(rows, np.array([1, 1, 1, 0, 1, 1], bool), 6, 4, [1, 3]).tolist() == [0, 1, 2, 3, 4, 5]
