"""tests/kv_bulk.py against tests/kv_reference.py, slot by slot; no GPU."""
import numpy as np
import pytest

from tests import kv_bulk, kv_reference as ref


@pytest.mark.parametrize("H,d,P", [(2, 64, 16), (1, 128, 32), (3, 128, 64)])
def test_bulk_packing_equals_slot_by_slot(H, d, P):
    rng = np.random.default_rng(d + P)
    pages, N = 5, 70
    at = rng.permutation(pages * P)[:N]
    phys, row = at // P, at % P
    k, v = ref.bf16(rng.standard_normal((N, H, d))), ref.bf16(rng.standard_normal((N, H, d)) * 2.0 ** rng.integers(-140, 100, (N, H, 1)))
    k[0], v[1, 0, 5], k[2, -1, 40] = 0, np.nan, -np.inf
    got = rng.integers(0, 256, (pages, H, P, 9 * d // 8), dtype=np.uint8)
    want = got.copy()
    kv_bulk.put(got, phys, row, k, v)
    for n in range(N):
        for h in range(H):
            ref.pack_slot(want, phys[n], h, row[n], k[n, h], v[n, h])
    assert np.array_equal(got, want)
    for n, (x, y) in enumerate(zip(*kv_bulk.get(want, phys, row, d))):
        for h in range(H):
            a, b = ref.unpack_slot(want, phys[n], h, row[n], d)
            assert np.array_equal(x[h], a, equal_nan=True) and np.array_equal(y[h], b, equal_nan=True)
