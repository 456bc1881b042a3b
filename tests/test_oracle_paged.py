"""Pins of oracle.paged: hand-worked page tables, closed forms of the rotation, attention against
oracle.full_attention."""
import numpy as np
import pytest

import oracle
from oracle import paged


def test_page_tables_by_hand():
    # pages of 4: request 0 has 3 positions (page 9) and gets 2; request 1 has none and gets 5; request 2
    # has 4 (page 8) and gets none
    table = [[9, -1, -1], [-1, -1, -1], [8, -1, -1]]
    r = paged.page_tables([3, 0, 4], [2, 5, 0], [1, 2, 3, 4, 5], 4, table, 4, 9)
    assert r["block_table"].tolist() == [[9, 4, -1], [3, 2, -1], [8, -1, -1]]
    assert r["slots"].tolist() == [39, 16, 12, 13, 14, 15, 8, -1, -1]
    assert r["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, -1, -1]
    assert r["q_start"].tolist() == [0, 2, 7, 7]
    assert r["kv_len"].tolist() == [5, 5, 4] and r["n_free_out"].tolist() == [1]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, f, pos = rng.normal(size=(3, 2, 128)), np.array([1.0, 0.37, 0.001]), [0, 5, 70]
    y, _ = paged.norm_rotate(x, None, 1e-6, pos, f, interleaved, 1.5)
    a, b = (slice(0, 6, 2), slice(1, 6, 2)) if interleaved else (slice(0, 3), slice(3, 6))
    z = (x[..., a] + 1j * x[..., b]) * 1.5 * np.exp(1j * np.array(pos)[:, None, None] * f)
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, atol=1e-13)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(1, 1, 128)), rng.normal(size=(1, 1, 128))
    f = [500000.0 ** (-2 * i / 128) for i in range(64)]
    dots = [(paged.norm_rotate(q, None, 1, [p + 17], f)[0] * paged.norm_rotate(k, None, 1, [p], f)[0]).sum()
            for p in (0, 1000, 2 ** 30)]
    np.testing.assert_allclose(dots, dots[0], atol=1e-11)


def test_norm_gives_unit_mean_square_times_the_weight():
    rng = np.random.default_rng(3)
    w = rng.normal(size=128)
    y, _ = paged.norm_rotate(rng.normal(size=(4, 3, 128)) * 7, w, 1e-30, [0] * 4, [])
    np.testing.assert_allclose(np.mean((y / w) ** 2, -1), 1.0, rtol=1e-12)


def test_attention_of_single_tokens_is_full_attention():
    rng = np.random.default_rng(4)
    K, V, Q = rng.normal(size=(2, 32, 128)), rng.normal(size=(2, 32, 128)), rng.normal(size=(2, 3, 128))
    pools = [np.stack([x[:, 16:], x[:, :16]]) for x in (K, V)]     # pages of 16, in the other order
    out, lse, _ = paged.attention(Q.reshape(1, 6, 128), *pools, [[1, 0]], [0, 1], [32])
    np.testing.assert_allclose(out[0].reshape(2, 3, 128), oracle.full_attention(Q, K, V), atol=1e-12)
    x = Q[1, 2] @ K[1].T / np.sqrt(128)
    np.testing.assert_allclose(lse[0, 5], np.log(np.exp(x).sum()), atol=1e-12)


def test_attention_masks_and_empty_rows():
    rng = np.random.default_rng(5)
    k, v, q = (rng.normal(size=s) for s in ((2, 1, 16, 128), (2, 1, 16, 128), (5, 1, 128)))
    out, lse, _ = paged.attention(q, k, v, [[1, 0]], [0, 4], [2])
    assert (out[:2] == 0).all() and (lse[:2, 0] == -np.inf).all()   # positions -2 and -1 see nothing
    np.testing.assert_allclose(out[2, 0], v[1, 0, 0])               # position 0 sees its own row only
    assert np.isfinite(out[3]).all() and np.isnan(out[4]).all()     # behind the last request: nothing
    v2 = v.copy()
    v2[1, 0, 1, 7] = np.inf                                         # position 1
    out2, _, _ = paged.attention(q, k, v2, [[1, 0]], [0, 4], [2])
    np.testing.assert_array_equal(out2[:3], out[:3])
    assert out2[3, 0, 7] == np.inf and np.isfinite(np.delete(out2[3, 0], 7)).all()


def test_gather_by_hand():
    pool = np.arange(3 * 1 * 16 * 128.0).reshape(1, 3, 1, 16, 128)
    got = paged.gather(pool, [[2, 0], [1, -1]], [20, 3], 2, 17)
    assert got.shape == (2, 1, 1, 17, 128)
    np.testing.assert_array_equal(got[0, 0, 0, :14], pool[0, 2, 0, 2:])
    np.testing.assert_array_equal(got[0, 0, 0, 14:], pool[0, 0, 0, :3])
    np.testing.assert_array_equal(got[1, 0, 0, 0], pool[0, 1, 0, 2])
    assert (got[1, 0, 0, 1:] == 0).all()
