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


@pytest.mark.parametrize("rotary,interleaved,n_axes,norm,n", [
    *[(r, i, a, w, n) for r, i in ((128, False), (128, True), (64, False), (96, True)) for a, w in ((2, True), (3, False), (4, True))
      for n in (1, 60)],
    (8, False, 2, True, 2600), (8, True, 3, False, 700)])
def test_write_axes_without_slots(wi, rotary, interleaved, n_axes, norm, n):
    """Keys and values to rows of their own instead of pages; tolerances as with slots (tests/test_gpu_paged8.py)."""
    rng = np.random.default_rng(rotary + n_axes + n)
    hq, hkv = 6, 2
    axis = [int(a) for a in rng.integers(0, n_axes, rotary // 2)]
    axis[0] = n_axes - 1
    x, X = bf(rng.normal(size=(n, hq + 2 * hkv, 128)))
    pos = rng.integers(-1000, 1 << 20, (n_axes, n))
    pos[0] = np.abs(pos[0])
    pad = np.arange(n) % 50 == 7
    pos[0, pad] = -1
    w, W = bf(1 + 0.3 * rng.normal(size=128))
    weights = (w, w) if norm else (None, None)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, 16, 1, 1, 1, rotary_dim=rotary, interleaved=interleaved), axes=axis)
    k, v = (torch.full((n, hkv, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    pc.write(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], i32(pos), None, k, v, q, *weights)
    pc.check()
    for got, part in ((f64(q), X[:, :hq]), (f64(k), X[:, hq:hq + hkv])):
        ref, normed = turned(part, W if norm else None, 1e-6, pos, freqs(rotary), axis, interleaved)
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * pair_size(normed, rotary, interleaved)
        assert (np.abs(got - ref) <= tol)[~pad].all()
        assert (got[pad] == 7).all()
    np.testing.assert_array_equal(f64(v)[~pad], X[~pad, hq + hkv:])
    assert (f64(v)[pad] == 7).all()
    # the same rows as the write into pages gives, in place of the queries
    page = 64
    slots = rng.permutation(-(-n // page) * page)[:n]
    paged = wi.PagedCache(wi.make_paged_config(hq, hkv, page, -(-n // page), 1, 1, rotary_dim=rotary,
                                               interleaved=interleaved), axes=axis)
    kp, vp = (torch.full((-(-n // page), hkv, page, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    own = x[:, :hq].contiguous()
    paged.write(own, x[:, hq:hq + hkv], x[:, hq + hkv:], i32(pos), i32(slots), kp, vp, own, *weights)
    paged.check()
    assert torch.equal(own[~torch.from_numpy(pad)], q[~torch.from_numpy(pad)])
    for rows, pool in ((k, kp), (v, vp)):
        assert torch.equal(rows, pool.transpose(1, 2).reshape(-1, hkv, 128)[torch.from_numpy(slots).to(DEV)])
    pc.free()
    paged.free()
