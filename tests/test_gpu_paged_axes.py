"""Positions of several axes on the GPU: the calls that tests/test_gpu_paged8.py's tests of axes do not make."""
import numpy as np
import pytest
import torch

from test_gpu_paged import DEV, bf, f64, freqs, i32
from test_gpu_paged8 import pair_size, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wi():
    import clustered_sparse_kv_gb300 as m
    return m


def test_one_axis_takes_positions_of_either_shape(wi):
    """axes that are all 0: positions [1][n], as of any number of axes, or [n], as of a cache without axes."""
    rng = np.random.default_rng(1)
    n, hq, hkv, page = 37, 4, 2, 16
    x, _ = bf(rng.normal(size=(n, hq + 2 * hkv, 128)))
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    pos, slots = i32(rng.integers(0, 5000, n)), i32(rng.permutation(4 * page)[:n])
    results = []
    for axes, shape in ((None, (n,)), (None, (1, n)), ([0] * 64, (n,)), ([0] * 64, (1, n))):
        pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, 4, 1, 1), axes=axes)
        pools = [torch.zeros((4, hkv, page, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        pools8 = [torch.zeros((4, hkv, page, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
        pools8 += [torch.zeros((4, hkv, 1), dtype=torch.uint8, device=DEV) for _ in range(2)]
        q = pc.write(*parts, pos.view(shape), slots, *pools)
        q8 = pc.write8(*parts, pos.view(shape), i32(np.arange(n)), *pools8)
        for bad in (pos.expand(2, n).contiguous(), pos.view(n, 1), pos.view(1, 1, n), pos[:n - 1], pos.cpu(), None):
            with pytest.raises(ValueError, match="positions"):
                pc.write(*parts, bad, slots, *pools)
        pc.check()
        pc.free()
        results.append([q, q8, *pools, *pools8])
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
