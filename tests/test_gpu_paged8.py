"""The paged cache in 8 bits, and rotations by several axes, on the GPU against oracle.paged (float64).

Tolerances.  Queries of the write: those of tests/test_gpu_paged.py (half a bf16 step, and 2^-19 of |a| + |b| for the fp32
terms of a rotated pair).  A value in 8 bits is off by at most half a step, 2^-4 of itself, or 2^-10 of its group's scale where
that is more; keys also by 2^-19 of |a| + |b| in front of the rounding.  Values (not rotated), copies and scales of values
are equal; a key's scale is that of its group's largest key, known to 2^-18.
Attention, on the pools' own bytes: a bf16 output is off by at most 2^-8 of itself; its weights by 2^-10, that is 2^-10 of
sum w|v|; a score is an fp32 dot of 128 products of the key with a query whose elements are known to 2^-17 of its largest
(two e4m3 pieces, the largest element scaled to 2^7 .. 2^8: half the smallest step, 2^-10, over 2^7): off by 128 * 2^-24 of
|q||k| / sqrt(128) and by sqrt(128) 2^-17 max|q| |k| / sqrt(128), and its weight by as much, once itself and once through the
sum; weights below 2^-27 of the row's largest may be missing, and the sums over n positions are fp32: n * 2^-24.
lse: the score's error, and n * 2^-24 of the sum.
"""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import DEV, bf, f64, freqs, i32, lay_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wi():
    import clustered_sparse_kv_gb300 as m
    return m


def values8(t):
    """The numbers of an e4m3 tensor."""
    return f64(t.view(torch.float8_e4m3fn).float())


def exps8(t):
    return t.view(torch.uint8).cpu().numpy().astype(np.int64) - 127


def as_values(x):
    """e4m3 tensor on the device of numbers that are e4m3's."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.float8_e4m3fn)
    assert np.array_equal(t.double().numpy(), np.asarray(x, np.float64), equal_nan=True)
    return t.to(DEV)


def as_scales(e):
    return torch.from_numpy((np.asarray(e) + 127).astype(np.uint8)).to(DEV).view(torch.float8_e8m0fnu)


def random_pool(rng, n_pages, hkv, page, scale=1.0, spread=1.0):
    """(values, exponents) of rows of a common direction and noise, of another size in every group."""
    size = np.exp(spread * rng.normal(size=(n_pages, hkv, page // 16, 1, 1))) * scale
    x = rng.normal(size=(n_pages, hkv, page // 16, 16, 128)) + rng.normal(size=(hkv, 1, 1, 128))
    x = x * size
    e = np.vectorize(paged.exponent)(np.abs(x).max((-1, -2)))
    return paged.e4m3(np.ldexp(x, -e[..., None, None])).reshape(n_pages, hkv, page, 128), e


def upload(pool):
    return as_values(pool[0]), as_scales(pool[1])


# ------------------------------------------------------------------ write ----

def turned(x, w, eps, pos, f, axis, interleaved, scale=1.0):
    """paged.norm_rotate with a position per axis: the pairs of one axis turn at a time."""
    pos = np.asarray(pos)
    if axis is None:
        return paged.norm_rotate(x, w, eps, pos, f, interleaved, scale)
    y, normed = paged.norm_rotate(x, w, eps, pos[0] * 0, f, interleaved, 1.0)
    for a in range(len(pos)):
        z, _ = paged.norm_rotate(x, w, eps, pos[a], f, interleaved, scale)
        for i in np.nonzero(np.asarray(axis) == a)[0]:
            for d in ((2 * i, 2 * i + 1) if interleaved else (i, i + len(f))):
                y[..., d] = z[..., d]
    return y, normed


def pair_size(normed, rotary, interleaved, scale=1.0):
    """|a| + |b| of the pair that an element turns in."""
    size, h = np.abs(normed), rotary // 2
    if rotary:
        a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, h), slice(h, rotary))
        both = (size[..., a] + size[..., b]) * max(abs(scale), 1)
        size[..., a] = size[..., b] = both
    return size


def write8_case(wi, new, ctx, hq, hkv, page, rotary=128, interleaved=False, norm=True, axis=None, seed=0, pad=0, scale=1.0,
                layout="fused", hole=None, grow=1.0):
    rng = np.random.default_rng(seed)
    kv = [c + n for c, n in zip(ctx, new)]
    table, n_pages = lay_out(kv, page, rng)
    live, total = sum(new), sum(new) + pad
    fused, F = bf(rng.normal(size=(total, hq + 2 * hkv, 128)) * rng.choice([0.01, 1, 30], size=(total, 1, 1)) * grow)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    if layout == "separate":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    Q, K, V = F[:, :hq], F[:, hq:hq + hkv], F[:, hq + hkv:]
    at = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)] + [[]]).astype(int)
    who = np.repeat(np.arange(len(new)), new)
    slots = np.full(total, -1)
    slots[:live] = table[who, at // page] * page + at % page
    if hole is not None and live > hole:
        slots[hole] = -1          # its query is wanted alone; the run is cut there
    n_axes = 1 if axis is None else max(axis) + 1
    pos = rng.integers(-300, 5000, (n_axes, total))
    pos[0, :live] = at
    pos[0, live:] = -1
    wq, WQ = bf(1 + rng.normal(size=128) * 0.3)
    wk, WK = bf(1 + rng.normal(size=128) * 0.3)
    f, eps = freqs(rotary) if rotary else [], 1e-5
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, len(new), table.shape[1], rotary_dim=rotary,
                                            interleaved=interleaved, inv_freq=f, eps=eps, rope_scale=scale), axes=axis)
    pools = [random_pool(rng, n_pages, hkv, page) for _ in range(2)]
    (kp, ks), (vp, vs) = (upload(p) for p in pools)
    out = torch.full((total, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    pc.write8(q, k, v, i32(pos if n_axes > 1 else pos[0]), i32(slots), kp, vp, ks, vs, out, wq if norm else None,
              wk if norm else None)
    pc.check()
    where = pos[:, :live] if axis is not None else pos[0, :live]
    rq, nq = turned(Q[:live], WQ if norm else None, eps, where, f, axis, interleaved, scale)
    rk, nk = turned(K[:live], WK if norm else None, eps, where, f, axis, interleaved, scale)
    got = f64(out)
    err = np.abs(got[:live] - rq)
    tol = 2.0 ** -8 * np.abs(rq) + (1 + 2.0 ** -8) * 2.0 ** -19 * pair_size(nq, rotary, interleaved, scale) + 2.0 ** -133
    assert (err <= tol).all(), (err / tol).max()
    assert (got[live:] == 7).all()
    # values: the same numbers
    RV, EV = paged.append8(*pools[1], V[:live], slots[:live])
    np.testing.assert_array_equal(exps8(vs), EV)
    np.testing.assert_array_equal(values8(vp), RV)
    # keys: half a step, and what fp32 may be off in front of the rounding
    size = pair_size(nk, rotary, interleaved, scale)
    EK = exps8(ks)
    _, lo = paged.append8(*pools[0], np.sign(rk) * np.maximum(np.abs(rk) - 2.0 ** -18 * size, 0), slots[:live])
    _, hi = paged.append8(*pools[0], np.sign(rk) * (np.abs(rk) + 2.0 ** -18 * size), slots[:live])
    assert ((lo <= EK) & (EK <= hi)).all()
    GK = values8(kp)
    RK, _ = paged.append8(*pools[0], rk, slots[:live])
    flat = GK.transpose(0, 2, 1, 3).reshape(-1, hkv, 128)
    same = RK.transpose(0, 2, 1, 3).reshape(-1, hkv, 128)
    steps = np.repeat(EK, 16, -1).transpose(0, 2, 1).reshape(-1, hkv)   # exponent of a slot
    ref_e = np.repeat(paged.append8(*pools[0], rk, slots[:live])[1], 16, -1).transpose(0, 2, 1).reshape(-1, hkv)
    stored = np.nonzero(slots[:live] >= 0)[0]
    rows = slots[stored]
    wide = np.ldexp(flat[rows], steps[rows][..., None])
    tol = np.maximum(2.0 ** -4 * np.abs(rk[stored]), np.ldexp(1.0, steps[rows] - 10)[..., None])
    tol = tol + (1 + 2.0 ** -4) * 2.0 ** -19 * size[stored]
    err = np.abs(wide - rk[stored])
    assert (err <= tol).all(), (err / tol).max()
    rest = np.setdiff1d(np.arange(n_pages * page), rows)
    alike = (steps == ref_e)[rest]
    np.testing.assert_array_equal(flat[rest][alike], same[rest][alike])
    # a second time: nothing is rounded again, nothing moves
    before = [t.view(torch.uint8).clone() for t in (kp, vp, ks, vs)]
    pc.write8(q, k, v, i32(pos if n_axes > 1 else pos[0]), i32(slots), kp, vp, ks, vs, out, wq if norm else None,
              wk if norm else None)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (kp, vp, ks, vs)))
    pc.check()
    pc.free()


@pytest.mark.parametrize("rotary,interleaved", [(128, False), (128, True), (64, False), (64, True), (8, False), (8, True),
                                                (96, False), (120, True), (0, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_write8_rotations(wi, rotary, interleaved, norm):
    write8_case(wi, [20, 1], [3, 40], 6, 2, 16, rotary, interleaved, norm, seed=rotary + interleaved)


@pytest.mark.parametrize("new,ctx", [([1], [0]), ([1], [1]), ([1], [15]), ([1], [16]), ([15], [0]), ([16], [0]), ([17], [0]),
                                     ([16], [5]), ([33], [14]), ([100], [47]), ([1] * 40, list(range(40))),
                                     ([3, 0, 20, 1, 50], [30, 5, 0, 47, 15])])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_write8_runs(wi, new, ctx, page):
    write8_case(wi, new, ctx, 4, 2, page, seed=len(new) + page, pad=3)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (28, 4), (32, 8), (5, 5), (8, 1), (6, 3), (40, 10)])
@pytest.mark.parametrize("layout", ["fused", "separate"])
def test_write8_heads(wi, hq, hkv, layout):
    write8_case(wi, [19, 1, 1], [7, 30, 47], hq, hkv, 16, seed=hq, layout=layout)


@pytest.mark.parametrize("ctx", [0, 5])
def test_write8_many_tokens(wi, ctx):
    write8_case(wi, [1500, 1, 700], [ctx, 31, 3 * ctx], 4, 2, 64, seed=3, pad=7)
    write8_case(wi, [3000], [ctx], 2, 2, 32, seed=4, norm=False, rotary=64, hole=1232 - ctx)


def test_write8_every_size_of_tile(wi):
    """Single tokens and chunks, of few tokens to more than 4096, which tiles of several sizes take."""
    write8_case(wi, [1] * 300, list(range(300)), 8, 8, 16, seed=20)
    write8_case(wi, [1] * 1000, [i % 50 for i in range(1000)], 8, 8, 16, seed=21)
    write8_case(wi, [1] * 500 + [700, 3, 40] + [1] * 99, [i % 33 for i in range(602)], 8, 8, 16, seed=22, pad=3)
    write8_case(wi, [1] * 400 + [3000, 17, 1000] + [2] * 99, [i % 33 for i in range(502)], 8, 8, 16, seed=23)


@pytest.mark.parametrize("hole", [0, 15, 16, 31, 39])
def test_write8_token_without_a_slot(wi, hole):
    """A token without a slot, the first or the last of its group: the rest of the group is written without it."""
    write8_case(wi, [40], [16], 4, 2, 16, seed=5, hole=hole)


@pytest.mark.parametrize("axis", [[0] * 16 + [1] * 24 + [2] * 24, [i % 3 for i in range(64)], [1] * 32 + [0] * 32, [3] * 64])
def test_write8_axes(wi, axis):
    write8_case(wi, [21, 1, 300], [3, 47, 0], 4, 2, 16, seed=6, axis=axis)
    write8_case(wi, [21, 1, 300], [3, 47, 0], 4, 2, 16, seed=7, axis=axis, interleaved=True, scale=1.3)


def test_write8_scale_and_large_values(wi):
    write8_case(wi, [20], [3], 4, 2, 16, seed=8, scale=0.7)
    write8_case(wi, [20], [3], 4, 2, 16, seed=9, norm=False, grow=1e35, rotary=0)
    write8_case(wi, [20], [3], 4, 2, 16, seed=10, norm=False, grow=1e-24, rotary=0)


def test_write8_infinities_nan_and_zeros(wi):
    rng = np.random.default_rng(11)
    x = rng.normal(size=(16, 1, 128))
    x[2, 0, 5], x[3, 0, 6], x[4, 0, 7], x[5] = np.inf, -np.inf, np.nan, 0.0
    t, X = bf(x)
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 3, 1, 1, rotary_dim=0))
    pools = [(np.zeros((3, 1, 16, 128)), np.zeros((3, 1, 1), int))] * 2
    (kp, ks), (vp, vs) = (upload(p) for p in pools)
    q = torch.ones((16, 1, 128), dtype=torch.bfloat16, device=DEV)
    pc.write8(q, t, t, i32(np.arange(16)), i32(np.arange(16) + 16), kp, vp, ks, vs)
    R, E = paged.append8(*pools[0], X, np.arange(16) + 16)
    for p, s in ((kp, ks), (vp, vs)):
        np.testing.assert_array_equal(exps8(s), E)
        np.testing.assert_array_equal(values8(p), R)
    # a group of zeros alone has the smallest scale; the next row is far above it
    z = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device=DEV)
    pc.write8(q[:1], z, z, i32([0]), i32([0]), kp, vp, ks, vs)
    assert exps8(ks)[0, 0, 0] == paged.LOWEST and (values8(kp)[0, 0, 0] == 0).all()
    pc.write8(q[:1], t[:1], t[:1], i32([0]), i32([1]), kp, vp, ks, vs)
    assert exps8(vs)[0, 0, 0] == paged.exponent(np.abs(X[0]).max()) and (values8(vp)[0, 0, 0] == 0).all()
    pc.check()
    pc.free()


def test_write8_reports_slots_outside_the_pool(wi):
    pc = wi.PagedCache(wi.make_paged_config(2, 1, 16, 2, 1, 1))
    x = torch.ones((3, 4, 128), dtype=torch.bfloat16, device=DEV)
    kp, vp = (torch.full((2, 1, 16, 128), 3, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((2, 1, 1), 100, dtype=torch.uint8, device=DEV) for _ in range(2))
    out = pc.write8(x[:, :2], x[:, 2:3], x[:, 3:], i32([0, 1, 2]), i32([31, 32, 0]), kp, vp, ks, vs)
    with pytest.raises(wi.WiError, match="page or slot"):
        pc.check()
    # the group of slot 0 begins anew; slot 31 continues one whose scale was 2^-27, and its rows in front, 3 * 2^-9 of that,
    # are nothing at the new one
    assert (kp.view(-1, 128)[1:16] == 3).all() and (kp.view(-1, 128)[16:31] == 0).all() and out.isfinite().all()
    assert values8(vp)[0, 0, 0, 0] * 2.0 ** exps8(vs)[0, 0, 0] == 1.0
    pc.free()


@pytest.mark.parametrize("rotary,interleaved", [(128, False), (128, True), (64, False), (96, True)])
@pytest.mark.parametrize("n_axes", [2, 3, 4])
def test_write_axes(wi, rotary, interleaved, n_axes):
    rng = np.random.default_rng(rotary + n_axes)
    n, hq, hkv, page = 150, 6, 2, 48
    axis = [int(a) for a in rng.integers(0, n_axes, rotary // 2)]
    axis[0] = n_axes - 1
    x, X = bf(rng.normal(size=(n, hq + 2 * hkv, 128)))
    pos = rng.integers(-1000, 1 << 20, (n_axes, n))
    pos[0] = np.abs(pos[0])
    pos[0, 7] = -1
    w, W = bf(1 + 0.3 * rng.normal(size=128))
    slots = rng.permutation(4 * page)[:n]
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, 4, 1, 1, rotary_dim=rotary, interleaved=interleaved), axes=axis)
    kp, vp = (torch.full((4, hkv, page, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    pc.write(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], i32(pos), i32(slots), kp, vp, out, w, w)
    pc.check()
    live = np.setdiff1d(np.arange(n), [7])
    for got, part in ((f64(out), X[:, :hq]), (f64(kp).transpose(0, 2, 1, 3).reshape(-1, hkv, 128)[slots], X[:, hq:hq + hkv])):
        ref, normed = turned(part, W, 1e-6, pos, freqs(rotary), axis, interleaved)
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * pair_size(normed, rotary, interleaved)
        assert (np.abs(got - ref) <= tol)[live].all()
        assert (got[7] == 7).all()
    one = wi.PagedCache(wi.make_paged_config(hq, hkv, page, 4, 1, 1, rotary_dim=rotary, interleaved=interleaved))
    same = i32(np.broadcast_to(pos[:1], pos.shape))   # every axis the same position: the plain write's bits
    a = pc.write(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], same, i32(slots), kp, vp, torch.zeros_like(out), w, w)
    b = one.write(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], same[0], i32(slots), kp, vp, torch.zeros_like(out), w, w)
    assert torch.equal(a, b)
    with pytest.raises(ValueError, match="positions"):
        pc.write(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], i32(pos[0]), i32(slots), kp, vp, out, w, w)
    one.free()
    pc.free()


# ------------------------------------------------------------------ attention ----

def attention8_case(wi, hq, hkv, page, new, kv, seed, pad=0, scale=1.0, poison=None, want_lse=True, spread_of=1.0):
    rng = np.random.default_rng(seed)
    table, n_pages = lay_out(kv, page, rng)
    q_start = np.concatenate([[0], np.cumsum(new)])
    n = int(q_start[-1]) + pad
    q, Q = bf(rng.normal(size=(max(n, 1), hq, 128)) * scale)
    pools = [random_pool(rng, n_pages, hkv, page, spread=spread_of) for _ in range(2)]
    if poison is not None:
        poison(pools, table)
    (kp, ks), (vp, vs) = (upload(p) for p in pools)
    K, V = (paged.widened(*p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, len(kv), table.shape[1]))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV) if want_lse else None
    args = (q, kp, vp, ks, vs, i32(table), i32(q_start), i32(kv))
    pc.attention8(*args, out=out, lse=lse)
    pc.check()
    compare(f64(out), None if lse is None else f64(lse), Q, K, V, table, q_start, kv)
    again = torch.full_like(out, 7.0)
    pc.attention8(*args, out=again)        # same bits, with and without lse
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    pc.check()
    pc.free()


def compare(got, gl, Q, K, V, table, q_start, kv):
    live = slice(0, int(q_start[-1]))
    ref, rlse, spread = paged.attention(Q, K, V, table, q_start, kv)
    assert (got[q_start[-1]:] == 7).all()
    # what a row may see: the keys that its call's requests hold
    held = [paged.rows_of(K, table[b], h, int(n)) for b, n in enumerate(kv) for h in range(K.shape[1])]
    kmax = max([np.linalg.norm(np.where(np.isfinite(x), x, 0), axis=-1).max(initial=0.0) for x in held])
    qn, qm = np.linalg.norm(Q[live], axis=-1), np.abs(Q[live]).max(-1, initial=0.0)
    ds = 128 * 2.0 ** -24 * qn * kmax / np.sqrt(128) + 2.0 ** -17 * qm * kmax + 2.0 ** -20
    most = max([1, *kv])
    tol = (2.0 ** -8 * np.abs(ref[live]) +
           (1 + 2.0 ** -7) * spread[live] * (2.0 ** -10 + 2 * ds + 2 * most * 2.0 ** -24)[..., None] + 2.0 ** -80)
    # a weight that is missing may belong to any value: the largest
    vmax = max([np.abs(np.where(np.isfinite(x), x, 0)).max(initial=0.0) for x in
                [paged.rows_of(V, table[b], h, int(n)) for b, n in enumerate(kv) for h in range(V.shape[1])]])
    tol = tol + most * 2.0 ** -27 * vmax
    good = np.isfinite(ref[live])
    err = np.abs(np.where(good, got[live], 0) - np.where(good, ref[live], 0))
    if err.size:
        assert (err[good] <= tol[good]).all(), (err[good] / tol[good]).max()
        np.testing.assert_array_equal(got[live][~good], ref[live][~good])
    if gl is not None:
        assert (gl[q_start[-1]:] == 7).all()
        same = gl[live] == rlse[live]     # -infinity where a row sees nothing
        ltol = ds + most * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(rlse[live]), rlse[live], 0)) + 2.0 ** -20
        with np.errstate(invalid="ignore"):
            assert (same | (np.abs(gl[live] - rlse[live]) <= ltol) | (np.isnan(gl[live]) & np.isnan(rlse[live]))).all()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 1), (10, 2), (6, 1), (28, 4), (8, 1), (32, 8)])
@pytest.mark.parametrize("new,ctx", [(1, 200), (5, 0), (19, 300), (70, 61)])
def test_attention8_heads(wi, hq, hkv, new, ctx):
    attention8_case(wi, hq, hkv, 16, [new], [ctx + new], seed=hq + new)


@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 383, 1000, 4097])
@pytest.mark.parametrize("page", [16, 48, 128, 8192])
def test_attention8_single_token_lengths(wi, kv, page):
    attention8_case(wi, 8, 2, page, [1], [kv], seed=kv)


@pytest.mark.parametrize("new", [1, 2, 3, 4, 5, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 260, 700])
@pytest.mark.parametrize("ctx", [0, 1, 100, 128, 515])
def test_attention8_chunk_lengths(wi, new, ctx):
    attention8_case(wi, 4, 1, 64, [new], [ctx + new], seed=new + ctx)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 96, 112, 128, 256, 1024, 1040])
def test_attention8_page_sizes(wi, page):
    attention8_case(wi, 4, 2, page, [40, 1, 130], [700, 333, 131], seed=page)
    attention8_case(wi, 4, 2, page, [1, 1, 1], [700, 333, 1], seed=page)


@pytest.mark.parametrize("seed", range(8))
def test_attention8_mixed_requests(wi, seed):
    rng = np.random.default_rng(100 + seed)
    hq, hkv = [(28, 4), (8, 2), (6, 1), (16, 8), (5, 1), (4, 4), (32, 8), (3, 3)][seed]
    batch = int(rng.integers(2, 30))
    new = rng.choice([0, 1, 1, 1, 2, 7, 40, 150], size=batch)
    ctx = rng.choice([0, 0, 3, 16, 127, 500, 1300, 2000], size=batch)
    attention8_case(wi, hq, hkv, int(rng.choice([16, 48, 64])), list(new), list(ctx + new), seed, pad=int(seed % 3))


@pytest.mark.parametrize("seed", range(6))
def test_attention8_batches_of_single_tokens(wi, seed):
    """One token or none of each request, the serving step."""
    rng = np.random.default_rng(200 + seed)
    hq, hkv = [(28, 4), (8, 2), (1, 1), (16, 8), (5, 1), (8, 1)][seed]
    batch = int(rng.integers(2, 90))
    new = rng.choice([0, 1, 1, 1], size=batch)
    kv = rng.choice([1, 3, 16, 127, 128, 500, 1300, 5000], size=batch)
    attention8_case(wi, hq, hkv, int(rng.choice([16, 48, 64])), list(new), list(kv), seed, pad=int(seed % 3))


def test_attention8_long_single_tokens(wi):
    attention8_case(wi, 8, 2, 16, [1, 1, 1], [30001, 5, 12000], seed=1)


def test_attention8_many_short_requests(wi):
    rng = np.random.default_rng(3)
    attention8_case(wi, 4, 2, 16, [1] * 700, list(rng.integers(1, 40, 700)), seed=2)


def test_attention8_large_scores(wi):
    """Scores of a few hundred: the running maximum moves far, and most weights are zero."""
    attention8_case(wi, 4, 2, 16, [90, 1], [600, 900], seed=4, scale=30.0)
    attention8_case(wi, 4, 2, 16, [1, 1], [600, 900], seed=4, scale=30.0)


def test_attention8_groups_of_very_different_size(wi):
    """Scales that differ by many powers of two, of keys and of values."""
    attention8_case(wi, 4, 2, 16, [90, 1], [600, 900], seed=4, spread_of=4.0, scale=0.05)
    attention8_case(wi, 4, 2, 16, [1, 1], [600, 900], seed=5, spread_of=4.0, scale=0.05)


def test_attention8_rows_that_see_nothing(wi):
    attention8_case(wi, 4, 1, 16, [10, 300, 1, 200], [3, 100, 0, 0], seed=5)
    attention8_case(wi, 28, 4, 16, [1, 1, 40], [0, 1, 39], seed=6)
    attention8_case(wi, 8, 2, 16, [1, 1, 1], [0, 1, 0], seed=6)


def test_attention8_no_tokens(wi):
    attention8_case(wi, 4, 1, 16, [0, 0], [50, 0], seed=7, pad=4)


@pytest.mark.parametrize("new,ctx", [([1], [20]), ([40], [0]), ([150, 1, 9], [90, 300, 119]), ([300], [1]), ([1, 1], [33, 700])])
def test_attention8_poison_behind_the_last_position(wi, new, ctx):
    """NaN behind the last position and in pages that no request holds, and scales of 2^127 there."""
    kv = [n + c for n, c in zip(new, ctx)]

    def poison(pools, table):
        for v, e in pools:
            page = v.shape[2]
            other = np.setdiff1d(np.arange(len(v)), table[table >= 0])
            v[other] = np.nan
            e[other] = 127
            for b, n in enumerate(kv):
                j, r = divmod(n, page)
                if r:
                    v[table[b, j], :, r:] = np.nan
                    e[table[b, j], :, -(-r // 16):] = 127

    attention8_case(wi, 8, 2, 16, new, kv, seed=8, poison=poison)
    attention8_case(wi, 8, 2, 128, new, kv, seed=8, poison=poison)


@pytest.mark.parametrize("hq,hkv", [(4, 1), (7, 1), (1, 1)])
@pytest.mark.parametrize("at", [130, 200, 259])
def test_attention8_poison_at_later_positions(wi, hq, hkv, at):
    """NaN of a later token reaches the tokens that see it and no others."""
    rng = np.random.default_rng(9)
    new, kv = [160, 1], [260, 50]
    table, n_pages = lay_out(kv, 16, rng)
    q, _ = bf(rng.normal(size=(161, hq, 128)))
    pools = [random_pool(rng, n_pages, hkv, 16) for _ in range(2)]
    clean = [upload(p) for p in pools]
    pools[0][0][table[0, at // 16], :, at % 16, 5] = np.nan
    pools[1][0][table[0, at // 16], :, at % 16, 9] = np.nan
    dirty = [upload(p) for p in pools]
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, 16, n_pages, 2, table.shape[1]))
    args = (i32(table), i32([0, 160, 161]), i32(kv))
    a, b = (pc.attention8(q, x[0][0], x[1][0], x[0][1], x[1][1], *args) for x in (clean, dirty))
    pc.check()
    sees = at - 100
    assert torch.equal(a[:sees], b[:sees]) and torch.equal(a[160], b[160])
    assert b[sees:160].isnan().all()      # through the score, every element
    pc.free()


@pytest.mark.parametrize("at", [30, 128, 141, 259])
def test_attention8_poison_in_a_value_alone(wi, at):
    """A NaN element of a token's value: in the rows that see it that element and no other, in the rest nothing."""
    def poison(pools, table):
        pools[1][0][table[0, at // pools[1][0].shape[2]], :, at % pools[1][0].shape[2], 9] = np.nan

    attention8_case(wi, 4, 1, 16, [260], [260], seed=10, poison=poison)
    attention8_case(wi, 7, 1, 64, [200, 1], [260, 70], seed=10, poison=poison)
    attention8_case(wi, 7, 1, 64, [1, 1], [260, 70], seed=10, poison=poison)


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("new", [[40, 3], [1, 1]])
def test_attention8_rows_do_not_touch_each_other(wi, value, new):
    """A query with an infinite or NaN element: NaN in its own row, nothing in the others, and nothing from queries
    behind the last token."""
    rng = np.random.default_rng(12)
    kv = [n + 200 for n in new]
    table, n_pages = lay_out(kv, 16, rng)
    n = sum(new)
    q, _ = bf(rng.normal(size=(n + 2, 8, 128)))
    (kp, ks), (vp, vs) = (upload(random_pool(rng, n_pages, 2, 16)) for _ in range(2))
    pc = wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, 2, table.shape[1]))
    args = (kp, vp, ks, vs, i32(table), i32([0, new[0], n]), i32(kv))
    a = pc.attention8(q, *args)
    p = q.clone()
    p[0, 3, 17] = value
    p[n:] = value
    b = pc.attention8(p, *args)
    pc.check()
    assert b[0, 3].isnan().all() and (b[n:] == 0).all()
    b[0, 3] = a[0, 3]
    assert torch.equal(a, b)
    pc.free()


def test_attention8_reports_bad_tables(wi):
    rng = np.random.default_rng(12)
    pc = wi.PagedCache(wi.make_paged_config(4, 1, 16, 8, 2, 4))
    q, _ = bf(rng.normal(size=(3, 4, 128)))
    (k, ks), (v, vs) = (upload(random_pool(rng, 8, 1, 16)) for _ in range(2))
    good = [[1, 2, 3, -1], [4, 5, -1, -1]]
    for starts in ([0, 2, 3], [0, 1, 2]):
        ref = pc.attention8(q, k, v, ks, vs, i32(good), i32(starts), i32([40, 20]))
        pc.check()
        a, b = list(range(starts[1])), list(range(starts[1], starts[2]))
        for table, start, kv, match, intact in [
                ([[1, 8, 3, -1], [4, 5, -1, -1]], starts, [40, 20], "page or slot", b),
                ([[1, 2, 3, -1], [4, -1, -1, -1]], starts, [40, 20], "page or slot", a),
                (good, starts, [40, 65], "length", a),
                (good, starts, [-1, 20], "length", b),
                (good, [0, starts[1], 4], [40, 20], "length", a),
                (good, [0, starts[1], starts[1] - 1], [40, 20], "length", a)]:
            out = torch.full_like(q, 7.0)
            pc.attention8(q, k, v, ks, vs, i32(table), i32(start), i32(kv), out=out)
            with pytest.raises(wi.WiError, match=match):
                pc.check()
            assert torch.equal(out[intact], ref[intact]), (table, start, kv)
    pc.check()
    pc.free()


def test_beyond_32_bit_offsets(wi):
    """Pools of more than 2^32 values; a request whose pages lie at both ends."""
    hkv, page, n_pages = 2, 64, 270000      # 270000 * 2 * 64 * 128 values: 4.4 GB each
    k, v = (torch.empty((n_pages, hkv, page, 128), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.empty((n_pages, hkv, page // 16), dtype=torch.uint8, device=DEV) for _ in range(2))
    rng = np.random.default_rng(13)
    table = np.array([[n_pages - 1, 0, n_pages - 2, 131072]])
    pools = [random_pool(rng, 4, hkv, page) for _ in range(2)]
    for (x, s), p in zip(((k, ks), (v, vs)), pools):
        a, b = upload(p)
        x[table[0]], s[table[0]] = a.view(torch.uint8), b.view(torch.uint8)
    K, V = (paged.widened(*p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(4, hkv, page, n_pages, 1, 4))
    for new in (30, 1):
        q, Q = bf(rng.normal(size=(new, 4, 128)))
        out = pc.attention8(q, k, v, ks, vs, i32(table), i32([0, new]), i32([250]))
        compare(f64(out), None, Q, K, V, [[0, 1, 2, 3]], [0, new], [250])
    ko, vo = (torch.empty((1, 1, hkv, 100, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pc.gather8(k, v, ks, vs, i32(table), i32([250]), 120, ko, vo)
    np.testing.assert_array_equal(f64(ko), paged.gather(K[None], [[0, 1, 2, 3]], [250], 120, 100))
    np.testing.assert_array_equal(f64(vo), paged.gather(V[None], [[0, 1, 2, 3]], [250], 120, 100))
    slots = [int(table[0, p // page]) * page + p % page for p in (0, 144, 192)]     # the first of their groups
    x = torch.ones((3, hkv, 128), dtype=torch.bfloat16, device=DEV)
    q = torch.ones((3, 4, 128), dtype=torch.bfloat16, device=DEV)
    pc.write8(q, x, x * 2, i32([0, 0, 0]), i32(slots), k, v, ks, vs)
    pc.check()
    for s in slots:
        at, row = s // page, s % page
        assert (values8(k[at, :, row]) * 2.0 ** exps8(ks[at, :, row // 16])[:, None] == 1).all()
        assert (values8(v[at, :, row]) * 2.0 ** exps8(vs[at, :, row // 16])[:, None] == 2).all()
    pc.free()


# ------------------------------------------------------------------ gather ----

@pytest.mark.parametrize("batch,layers,hkv,page,pos0,n,kv_hi", [
    (1, 1, 1, 16, 0, 1, 1), (1, 1, 8, 16, 0, 300, 300), (3, 2, 2, 48, 17, 100, 160), (16, 3, 4, 16, 40, 1, 60),
    (2, 1, 3, 64, 0, 513, 400), (5, 2, 1, 1024, 999, 65, 2000), (1, 1, 2, 16, 200, 50, 100)])
def test_gather8(wi, batch, layers, hkv, page, pos0, n, kv_hi):
    rng = np.random.default_rng(batch + n)
    kv = rng.integers(0, kv_hi + 1, batch)
    kv[0] = kv_hi
    table, n_pages = lay_out(kv, page, rng)
    width = max(table.shape[1], -(-(pos0 + n) // page))
    table = np.concatenate([table, np.full((batch, width - table.shape[1]), -1)], 1)
    pools = []
    for _ in range(2):
        v, e = random_pool(rng, layers * n_pages, hkv, page, spread=8.0)
        v[rng.random(v.shape) < 0.01] = np.nan
        e[rng.random(e.shape) < 0.05] = -64
        pools.append((v.reshape(layers, n_pages, hkv, page, 128), e.reshape(layers, n_pages, hkv, page // 16)))
    (k, ks), (v, vs) = (upload(p) for p in pools)
    K, V = (paged.widened(*p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hkv, hkv, page, n_pages, batch, width))
    ko, vo = (torch.full((batch, layers, hkv, n, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pools = (k, v, ks, vs) if layers > 1 else (k[0], v[0], ks[0], vs[0])
    pc.gather8(*pools, i32(table), i32(kv), pos0, ko, vo)
    pc.check()
    np.testing.assert_array_equal(f64(ko), paged.gather(K, table, kv, pos0, n))
    np.testing.assert_array_equal(f64(vo), paged.gather(V, table, kv, pos0, n))
    pc.free()


def test_gather8_reports_bad_tables(wi):
    rng = np.random.default_rng(14)
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 4, 2, 2))
    (k, ks), (v, vs) = (upload(random_pool(rng, 4, 1, 16)) for _ in range(2))
    ko, vo = (torch.zeros((2, 1, 1, 20, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pc.gather8(k, v, ks, vs, i32([[0, 4], [1, 2]]), i32([20, 20]), 0, ko, vo)
    with pytest.raises(wi.WiError, match="page or slot"):
        pc.check()
    K = paged.widened(values8(k), exps8(ks))
    np.testing.assert_array_equal(f64(ko[1, 0]), paged.gather(K[None], [[1, 2]], [20], 0, 20)[0, 0])
    pc.gather8(k, v, ks, vs, i32([[0, 3], [1, 2]]), i32([33, 20]), 0, ko, vo)
    with pytest.raises(wi.WiError, match="length"):
        pc.check()
    pc.free()


# ------------------------------------------------------------------ together ----

def test_serving_steps_in_8_bits_then_index(wi):
    """Requests prefilled in chunks and decoded token by token through tables, write8 and attention8; then an index from
    the pages, which is that of the rows that gather8 gives."""
    rng = np.random.default_rng(15)
    hq, hkv, page, n_pages, width = 8, 2, 16, 400, 140
    f = freqs(128)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 2, width, inv_freq=f))
    kp, vp = (torch.full((n_pages, hkv, page, 128), 127, dtype=torch.uint8, device=DEV) for _ in range(2))   # NaN
    ks, vs = (torch.full((n_pages, hkv, 1), 254, dtype=torch.uint8, device=DEV) for _ in range(2))
    table = i32(np.full((2, width), -1))
    free, left = i32(rng.permutation(n_pages)), i32([n_pages])
    ctx = np.zeros(2, int)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    for new in ([1000, 37], [1040, 1], [1, 1], [1, 1], [6, 17], [1, 1]):
        n = sum(new) + 2
        kv, start, slots, pos, out_left = i32([0, 0]), i32([0] * 3), i32([0] * n), i32([0] * n), i32([0])
        pc.tables(i32(ctx), i32(new), free, left, table, kv, start, slots, pos, out_left)
        left = out_left
        x, _ = bf(rng.normal(size=(n, hq + 2 * hkv, 128)))
        q = pc.write8(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, kp, vp, ks, vs, None, w, w)
        out = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((n, hq), 7.0, device=DEV)
        pc.attention8(q, kp, vp, ks, vs, table, start, kv, out=out, lse=lse)
        pc.check()
        K, V = paged.widened(values8(kp), exps8(ks)), paged.widened(values8(vp), exps8(vs))
        compare(f64(out), f64(lse), f64(q), K, V, table.cpu().numpy(), start.cpu().numpy(), kv.cpu().numpy())
        ctx += new
    rows = [torch.empty((1, 1, hkv, 2048, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pc.gather8(kp, vp, ks, vs, table[:1].contiguous(), kv[:1], 0, *rows)
    cfg = wi.make_config(1, 1, hq, hkv, 2048, seg_len=1024, clusters_per_seg=64, iters=2)
    a = wi.WaveIndex.build_paged(cfg, pc, kp, vp, table[:1].contiguous(), kv[:1].contiguous(), k_scales=ks, v_scales=vs)
    b = wi.WaveIndex.build(cfg, *rows)
    q, _ = bf(rng.normal(size=(1, 1, hq, 128)))
    assert torch.equal(a.decode(q), b.decode(q))
    assert a.decode(q).isfinite().all()
    with pytest.raises(ValueError, match="together"):
        wi.WaveIndex.build_paged(cfg, pc, kp, vp, table[:1].contiguous(), kv[:1].contiguous(), k_scales=ks)
    for x in (a, b, pc):
        x.free()


def test_captured_step_in_8_bits_replays_over_new_contents(wi):
    """write8 and attention8 in one graph, replayed with other lengths, tables and rows."""
    rng = np.random.default_rng(16)
    hq, hkv, page, n_pages, width = 8, 2, 16, 200, 90
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 3, width))
    x = torch.zeros((3, hq + 2 * hkv, 128), dtype=torch.bfloat16, device=DEV)
    pools = [random_pool(rng, n_pages, hkv, page) for _ in range(2)]
    (kp, ks), (vp, vs) = (upload(p) for p in pools)
    table, kv, start = i32(np.zeros((3, width))), i32([0] * 3), i32([0] * 4)
    pos, slots = i32([0] * 3), i32([0] * 3)
    q = torch.zeros((3, hq, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(q)

    def step():
        pc.write8(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, kp, vp, ks, vs, q)
        pc.attention8(q, kp, vp, ks, vs, table, start, kv, out=out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lengths in ([5, 700, 1300], [1, 16, 17], [300, 301, 302]):
        t, _ = lay_out(lengths, page, rng)
        table.copy_(i32(np.pad(t, ((0, 0), (0, width - t.shape[1])), constant_values=-1)))
        kv.copy_(i32(lengths)), start.copy_(i32([0, 1, 2, 3]))
        at = np.array(lengths) - 1
        slots.copy_(i32(t[np.arange(3), at // page] * page + at % page)), pos.copy_(i32(at))
        x.copy_(bf(rng.normal(size=x.shape))[0])
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        pc.check()
        K, V = paged.widened(values8(kp), exps8(ks)), paged.widened(values8(vp), exps8(vs))
        compare(f64(out), None, f64(q), K, V, t, [0, 1, 2, 3], lengths)
    pc.free()


def test_calls_in_8_bits_refuse_bad_arguments(wi):
    pc = wi.PagedCache(wi.make_paged_config(4, 2, 32, 4, 2, 4))
    n = 3
    x = torch.zeros((n, 8, 128), dtype=torch.bfloat16, device=DEV)
    kp, vp = (torch.zeros((4, 2, 32, 128), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((4, 2, 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    ints = i32([0, 1, 2])
    out = torch.zeros((n, 4, 128), dtype=torch.bfloat16, device=DEV)
    ok = dict(q=q, k=k, v=v, positions=ints, slots=ints, k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, q_out=out)
    pc.write8(**ok)
    for bad in (dict(slots=None), dict(k_pages=kp.float()), dict(k_pages=kp.view(torch.float8_e5m2)), dict(k_scales=ks[:2]),
                dict(v_scales=vs.view(torch.float8_e4m3fn)), dict(k_scales=None), dict(k_pages=kp[:, :, :16]),
                dict(v_scales=vs.cpu()), dict(positions=i32([[0, 1, 2]] * 2)), dict(q_out=x[:, :4])):
        with pytest.raises(ValueError):
            pc.write8(**{**ok, **bad})
    for bad in (dict(k_pages=vp), dict(v_scales=ks), dict(k_scales=kp.view(-1)[:16].view(4, 2, 2))):
        with pytest.raises(wi.WiError, match="memory"):
            pc.write8(**{**ok, **bad})
    table, start, kv = i32(np.zeros((2, 4))), i32([0, 1, 3]), i32([5, 6])
    ok = dict(q=out, k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, block_table=table, q_start=start, kv_len=kv)
    pc.attention8(**ok)
    for bad in (dict(k_scales=ks[:2]), dict(v_pages=vp.to(torch.bfloat16)), dict(k_scales=None), dict(q=q), dict(kv_len=start)):
        with pytest.raises(ValueError):
            pc.attention8(**{**ok, **bad})
    with pytest.raises(wi.WiError, match="memory"):
        pc.attention8(**ok, out=out)
    rows = [torch.zeros((2, 1, 2, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ok = dict(k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, block_table=table, kv_len=kv, pos0=0, k_out=rows[0],
              v_out=rows[1])
    pc.gather8(**ok)
    for bad in (dict(k_scales=ks[None]), dict(k_out=rows[0].float()), dict(v_pages=vp[None])):
        with pytest.raises(ValueError):
            pc.gather8(**{**ok, **bad})
    with pytest.raises(wi.WiError, match="memory"):
        pc.gather8(**{**ok, "v_out": rows[0]})
    with pytest.raises(wi.WiError, match="positions"):
        pc.gather8(**{**ok, "pos0": 125})
    pc.check()
    pc.free()
    for bad in ([0] * 63, [], [4] * 64, [-1] + [0] * 63):
        with pytest.raises((ValueError, wi.WiError)):
            wi.PagedCache(wi.make_paged_config(4, 2, 32, 4, 2, 4), axes=bad)
