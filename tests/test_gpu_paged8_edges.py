"""Corners of the paged cache in 8 bits on the GPU: very long contexts, sinks of attention, references that move, bad offsets,
handles and streams.  Tolerances as tests/test_gpu_paged8.py derives them."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import DEV, bf, f64, i32, lay_out
from test_gpu_paged8 import as_scales, as_values, compare, exps8, random_pool, upload, values8
from test_gpu_paged_edges import repeated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wi():
    import clustered_sparse_kv_gb300 as m
    return m


# ------------------------------------------------------------ long contexts ----

@pytest.mark.parametrize("hq,hkv,new,kv", [
    (8, 2, [1] * 80, [1 << 20] * 80),                          # single tokens, whole in their CTAs
    (4, 1, [1], [(1 << 27) - 77]),                             # cut: every CTA adds up more than once
    (8, 1, [1], [(1 << 27) - 77]),
    (4, 1, [40], [(1 << 26) - 77]),                            # two tiles, cut
    (4, 1, [40] * 200, [(1 << 19) + 300] * 200),               # two tiles, whole or cut anywhere
    (8, 1, [1, 33, 2, 0, 16, 1, 70], [1 << 23, 3 << 20, 900, 5, (1 << 22) + 1, 7 << 20, 555555]),
])
def test_attention8_over_millions_of_positions(wi, hq, hkv, new, kv):
    """Long contexts over few distinct rows, which the 64-bit softmax counts instead of adding them one by one."""
    rng = np.random.default_rng(58)
    unique, tables = {}, []
    for n in kv:
        if n not in unique:
            unique[n] = repeated(n, rng)
        tables.append(unique[n][0])
    width = max(len(t) for t in tables)
    table = np.zeros((len(kv), width), np.int64)
    for b, t in enumerate(tables):
        table[b, :len(t)] = t
    start = np.concatenate([[0], np.cumsum(new)])
    n = int(start[-1])
    q, Q = bf(rng.normal(size=(n, hq, 128)))
    pools = [random_pool(rng, 8, hkv, 128, spread=0.3) for _ in range(2)]
    (k, ks), (v, vs) = (upload(p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, 128, 8, len(kv), width))
    lse = torch.empty((n, hq), device=DEV)
    args = (q, k, v, ks, vs, i32(table), i32(start), i32(kv))
    out = pc.attention8(*args, lse=lse)
    pc.check()
    again = pc.attention8(*args)
    pc.check()
    pc.free()
    assert torch.equal(out, again)
    out, lse = f64(out), f64(lse)
    K, V = (paged.widened(*p).transpose(1, 0, 2, 3).reshape(hkv, -1, 128) for p in pools)
    for b in range(len(kv)):
        if b >= 8 and b % 37:       # requests alike: some are enough
            continue
        row = unique[kv[b]][1]
        counts = np.bincount(row[:max(kv[b] - new[b], 0)], minlength=1024).astype(np.float64)
        for i in range(new[b]):
            p, t = kv[b] - new[b] + i, start[b] + i
            counts[row[p]] += 1
            for h in range(hq):
                x = K[h // (hq // hkv)] @ Q[t, h] / np.sqrt(128)
                w = counts * np.exp(x - x.max())
                z = w.sum()
                ref, spread = w / z @ V[h // (hq // hkv)], w / z @ np.abs(V[h // (hq // hkv)])
                # weights to 2^-10, the result rounded to bf16, 2^-8; a score is off by ds, and its weight by as much, once itself
                # and once through the sum; a segment's additions as in the bf16 attention, 2^-8, the sums of a row less
                kn = np.linalg.norm(K[h // (hq // hkv)], axis=1).max()
                ds = 128 * 2.0 ** -24 * np.linalg.norm(Q[t, h]) * kn / np.sqrt(128) + 2.0 ** -17 * np.abs(Q[t, h]).max() * kn
                assert (np.abs(out[t, h] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10 + 2 * ds) * spread).all()
                assert abs(lse[t, h] - (np.log(z) + x.max())) <= ds + 2.0 ** -12


@pytest.mark.parametrize("batch,new", [(2 * 152, 1), (152, 40)])
def test_attention8_adds_long_contexts_up_in_parts(wi, batch, new):
    """Equal scores over values of one sign: what the additions lose does not grow with the context.  A bf16 rounding, and
    2^-8 for the additions."""
    rng = np.random.default_rng(59)
    kv = 1 << 22
    table, row = repeated(kv, rng)
    values = paged.e4m3(rng.uniform(0.5, 1.5, size=(8, 1, 128, 128)))
    zero = np.zeros((8, 1, 8), int)
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 128, 8, batch, len(table)))
    q = torch.zeros((batch * new, 1, 128), dtype=torch.bfloat16, device=DEV)
    out = pc.attention8(q, as_values(values * 0), as_values(values), as_scales(zero), as_scales(zero),
                        i32(table)[None].repeat(batch, 1), i32(np.arange(batch + 1) * new), i32([kv] * batch))
    pc.check()
    pc.free()
    out = f64(out).reshape(batch, new, 128)
    for i in (0, new - 1):
        ref = np.bincount(row[:kv - new + i + 1], minlength=1024) / (kv - new + i + 1) @ values.reshape(1024, 128)
        assert (np.abs(out[:, i] - ref) <= 2.0 ** -7 * ref).all()


@pytest.mark.parametrize("single", [True, False])
def test_attention8_over_a_quarter_of_a_billion_positions(wi, single):
    """Two million blocks of one item, in one CTA where there are as many items as CTAs.  One page holds every position;
    with equal scores and powers of two as values every sum is exact."""
    kv = 1 << 28
    n = 1 if single else 256 * torch.cuda.get_device_properties(0).multi_processor_count
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 128, 1, 1, kv // 128))
    V = np.broadcast_to(2.0 ** (np.arange(128) % 4), (1, 1, 128, 128))
    zero = np.zeros((1, 1, 8), int)
    q = torch.zeros((n, 1, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((n, 1), device=DEV)
    out = pc.attention8(q, as_values(V * 0), as_values(V), as_scales(zero), as_scales(zero),
                        torch.zeros((1, kv // 128), dtype=torch.int32, device=DEV), i32([0, n]), i32([kv]), lse=lse)
    pc.check()
    pc.free()
    assert (f64(out) == V[0, 0, 0]).all()
    assert (lse - 28 * np.log(2)).abs().max() < 2.0 ** -12       # the rows see 2^28 positions and up to n fewer


@pytest.mark.parametrize("hq,new", [(1, 300), (4, 40)])
def test_attention8_poison_where_a_long_context_is_cut(wi, hq, new):
    """NaN values on both sides of position 2^18, where the first 2048 blocks end, in the middle of the tokens' own
    positions: they reach the tokens that see them, in their two elements, and no others."""
    rng = np.random.default_rng(60)
    kv, batch, at = (1 << 18) + new // 2, 100, ((1 << 18) - 9, (1 << 18) + 3)
    table, row = repeated(kv, rng)
    table[-4:] = [8, 9, 10, 11]                 # the last blocks' pages are used once
    row = (table[:, None] * 128 + np.arange(128)).reshape(-1)[:kv]
    pools = [random_pool(rng, 12, 1, 128, spread=0.3) for _ in range(2)]
    flat = pools[1][0].reshape(-1, 128)
    flat[row[at[0]], 9], flat[row[at[1]], 70] = np.nan, np.nan
    q, Q = bf(rng.normal(size=(new, hq, 128)))
    (k, ks), (v, vs) = (upload(p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hq, 1, 128, 12, batch, len(table)))
    out = pc.attention8(q.repeat(batch, 1, 1), k, v, ks, vs, i32(table)[None].repeat(batch, 1),
                        i32(np.arange(batch + 1) * new), i32([kv] * batch))
    pc.check()
    pc.free()
    out = f64(out).reshape(batch, new, hq, 128)
    K, V = (paged.widened(*p).reshape(-1, 128) for p in pools)
    clean = np.where(np.isfinite(V), V, 0)
    counts = np.bincount(row[:kv - new], minlength=12 * 128).astype(np.float64)
    for i in range(new):
        p = kv - new + i
        counts[row[p]] += 1
        x = Q[i] @ K.T / np.sqrt(128)
        w = counts * np.exp(x - x.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        ref, spread = w @ clean, w @ np.abs(clean)
        got = out[:, i]
        if p >= at[0]:
            assert np.isnan(got[..., 9]).all(), i
        if p >= at[1]:
            assert np.isnan(got[..., 70]).all(), i
        fine = np.ones(128, bool)
        fine[[9] * (p >= at[0]) + [70] * (p >= at[1])] = False
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -8 * spread)[..., fine].all(), i


# ------------------------------------------------------------ weights far apart ----

@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("gap", [5.0, 9.0, 12.0, 17.0])
@pytest.mark.parametrize("where", [0, 3000, 19990])
def test_attention8_behind_a_sink(wi, new, gap, where):
    """One position that weighs e^gap as much as any other, with a value of nothing: what is left of the row is the sum of
    20000 weights of e^-gap, down to 2^-25 of the largest, and none of it may be lost."""
    rng = np.random.default_rng(61)
    kv, hq, page = 20000 + new, 4, 16
    table, n_pages = lay_out([kv], page, rng)
    base = np.full(128, np.sqrt(gap * np.sqrt(128) / 128))      # q . k of the sink: gap * sqrt(128)
    pools = [(np.zeros((n_pages, 1, page, 128)), np.full((n_pages, 1, 1), -6)) for _ in range(2)]
    K, V = pools[0][0], pools[1][0]
    for j, pg in enumerate(table[0]):
        K[pg, 0] = paged.e4m3(rng.normal(size=(page, 128)) * 0.05 * 64)
        V[pg, 0] = paged.e4m3((1 + 0.1 * rng.normal(size=(page, 128))) * 64)
    K[table[0, where // page], 0, where % page] = paged.e4m3(base * 64)
    V[table[0, where // page], 0, where % page] = 0
    q, Q = bf(np.broadcast_to(base, (new, hq, 128)))
    (k, ks), (v, vs) = (upload(p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hq, 1, page, n_pages, 1, table.shape[1]))
    out = torch.full((new, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((new, hq), 7.0, device=DEV)
    pc.attention8(q, k, v, ks, vs, i32(table), i32([0, new]), i32([kv]), out=out, lse=lse)
    pc.check()
    pc.free()
    K, V = (paged.widened(*p) for p in pools)
    ref, rlse, spread = paged.attention(Q, K, V, table, [0, new], [kv])
    assert (np.abs(ref) > 1e-4).all()
    # 2^-8 of the result, 2^-10 of the weights, the scores' 128 * 2^-24 * gap twice and 2^-17 max|q||k| twice (< 2^-12 each)
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2.0 ** -10) * spread).all()
    assert (np.abs(f64(lse) - rlse) <= 2.0 ** -11).all()


@pytest.mark.parametrize("order", ["rising", "falling", "late"])
@pytest.mark.parametrize("new", [1, 33])
def test_attention8_maxima_that_move_far(wi, order, new):
    """Scores that climb or fall by hundreds over a request: a row takes one reference after the other."""
    rng = np.random.default_rng(62)
    kv, hq, page = 3000, 4, 16
    table, n_pages = lay_out([kv], page, rng)
    base = rng.normal(size=128)
    base *= np.sqrt(128) / np.linalg.norm(base)
    level = {"rising": np.linspace(-10, 10, kv), "falling": np.linspace(10, -10, kv), "late": np.where(np.arange(kv) < 2900, -10, 10)}
    rows = base * level[order][:, None] + 0.2 * rng.normal(size=(kv, 128))
    K, V = np.zeros((n_pages, 1, page, 128)), rng.normal(size=(n_pages, 1, page, 128))
    for p in range(kv):
        K[table[0, p // page], 0, p % page] = rows[p]
    pools = []
    for x in (K, V):
        e = np.vectorize(paged.exponent)(np.abs(x).max((-1, -2)))[..., None]
        pools.append((paged.e4m3(np.ldexp(x, -e[..., None])), e))
    q, Q = bf(np.broadcast_to(base * 3, (new, hq, 128)) + 0.2 * rng.normal(size=(new, hq, 128)))
    (k, ks), (v, vs) = (upload(p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hq, 1, page, n_pages, 1, table.shape[1]))
    out = torch.full((new, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((new, hq), 7.0, device=DEV)
    pc.attention8(q, k, v, ks, vs, i32(table), i32([0, new]), i32([kv]), out=out, lse=lse)
    pc.check()
    pc.free()
    compare(f64(out), f64(lse), Q, *(paged.widened(*p) for p in pools), table, [0, new], [kv])


@pytest.mark.parametrize("new", [1, 33])
def test_attention8_values_of_very_different_scales(wi, new):
    """Groups whose values differ by 2^80 and more: what is small beside the largest is lost in the output, as it is in
    fp32, but not in the sum of the weights."""
    rng = np.random.default_rng(63)
    kv, hq, page = 1000, 4, 16
    table, n_pages = lay_out([kv], page, rng)
    k_pool = random_pool(rng, n_pages, 1, page, spread=0.3)
    values = paged.e4m3(rng.normal(size=(n_pages, 1, page, 128)) * 50)
    for exps in (rng.choice([-64, -10], (n_pages, 1, 1)), np.full((n_pages, 1, 1), -64), rng.choice([-60, 20, 40], (n_pages, 1, 1))):
        pools = [k_pool, (values, exps)]
        q, Q = bf(rng.normal(size=(new, hq, 128)) * 2)
        (k, ks), (v, vs) = (upload(p) for p in pools)
        pc = wi.PagedCache(wi.make_paged_config(hq, 1, page, n_pages, 1, table.shape[1]))
        out = torch.full((new, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((new, hq), 7.0, device=DEV)
        pc.attention8(q, k, v, ks, vs, i32(table), i32([0, new]), i32([kv]), out=out, lse=lse)
        pc.check()
        pc.free()
        compare(f64(out), f64(lse), Q, *(paged.widened(*p) for p in pools), table, [0, new], [kv])


# ------------------------------------------------------------ offsets, handles, streams ----

@pytest.mark.parametrize("start,good", [
    ([0, 5, 2, 5], 1),                  # request 2 alone would be fine, and write rows of request 0
    ([0, 5, 7, 3, 10, 12], 2),
    ([0, 12, 0, 12, 0, 12], 1),         # every other request claims all rows
    ([5, 4, 4, 12], 0),
    ([0, 3, 3, 12, 11], 3),
    ([0] + [6, 2] * 250, 1),            # in another thread's share of the requests
    ([0] * 450 + [7, 1, 9], 450),
])
def test_attention8_keeps_requests_apart_where_offsets_fall(wi, start, good):
    """The requests in front of a falling offset are answered as if they were the whole call; rows of none behind it."""
    rng = np.random.default_rng(53)
    n, batch = 12, len(start) - 1
    table, n_pages = lay_out([300], 16, rng)
    q = bf(rng.normal(size=(n, 8, 128)))[0]
    (k, ks), (v, vs) = (upload(random_pool(rng, n_pages, 2, 16)) for _ in range(2))
    pc = wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, max(batch, 1), table.shape[1]))
    table, kv = i32(table.repeat(batch, 0)), i32([300] * batch)
    outs, lses = ([torch.full(s, 7.0, dtype=t, device=DEV) for _ in range(2)]
                  for s, t in (((n, 8, 128), torch.bfloat16), ((n, 8), torch.float32)))
    if good:
        # as many requests as in the other call, so that the same kernel answers: those behind the good ones have no tokens
        rest = [start[good]] * (batch - good)
        pc.attention8(q, k, v, ks, vs, table, i32(start[:good + 1] + rest), kv, out=outs[0], lse=lses[0])
        pc.check()
    pc.attention8(q, k, v, ks, vs, table, i32(start), kv, out=outs[1], lse=lses[1])
    with pytest.raises(wi.WiError, match="length"):
        pc.check()
    assert torch.equal(*outs) and torch.equal(*lses)
    assert (outs[1][start[good]:] == 7).all() and (outs[1][start[0]:start[good]] != 7).any(-1).all()
    pc.free()


def test_attention8_calls_in_turn_and_on_two_streams(wi):
    """One handle used for single tokens and chunks, in 8 bits and in bf16 in turn, many times, and two handles at once on
    two streams: always the same bits."""
    rng = np.random.default_rng(35)
    kv = [3000, 2000, 700]
    table, n_pages = lay_out(kv, 16, rng)
    (k, ks), (v, vs) = (upload(random_pool(rng, n_pages, 2, 16)) for _ in range(2))
    kb, vb = (bf(rng.normal(size=(n_pages, 2, 16, 128)))[0] for _ in range(2))
    pcs = [wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, 3, table.shape[1])) for _ in range(2)]
    jobs = []
    for new in [(1, 0, 0), (1, 1, 1), (0, 200, 90), (2, 0, 0), (150, 1, 33)]:
        q = bf(rng.normal(size=(sum(new), 8, 128)))[0]
        tables = (i32(table), i32(np.concatenate([[0], np.cumsum(new)])), i32(kv))
        jobs.append(("attention8", (q, k, v, ks, vs, *tables)))
        jobs.append(("attention", (q, kb, vb, *tables)))
    first = [getattr(pcs[0], f)(*j) for f, j in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (f, j), o in zip(jobs, first):
            assert torch.equal(getattr(pcs[0], f)(*j), o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(f) for _ in range(10) for f in first] for _ in range(2)]
    for i in range(len(outs[0])):
        for s in range(2):
            n = i if s == 0 else len(outs[0]) - 1 - i   # different jobs at the same time
            f, j = jobs[n % len(jobs)]
            getattr(pcs[s], f)(*j, out=outs[s][n], stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        for n, o in enumerate(outs[s]):
            assert torch.equal(o, first[n % len(jobs)])
        pcs[s].check()
        pcs[s].free()


def test_written_groups_do_not_depend_on_what_stood_there(wi):
    """A group that a call begins takes nothing from its old rows and scale, NaN and 2^127 included; rows behind the last
    stay as they were, bit for bit."""
    rng = np.random.default_rng(64)
    pc = wi.PagedCache(wi.make_paged_config(4, 2, 32, 3, 1, 3))
    x = bf(rng.normal(size=(21, 8, 128)))[0]
    slots, pos = i32(np.arange(21) + 32), i32(np.arange(21))
    got = []
    for fill, scale in ((0, 0), (127, 254), (255, 255), (51, 130)):
        kp, vp = (torch.full((3, 2, 32, 128), fill, dtype=torch.uint8, device=DEV) for _ in range(2))
        ks, vs = (torch.full((3, 2, 2), scale, dtype=torch.uint8, device=DEV) for _ in range(2))
        pc.write8(x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, kp, vp, ks, vs)
        pc.check()
        for p, s in ((kp, ks), (vp, vs)):
            assert (p[[0, 2]] == fill).all() and (p[1, :, 21:] == fill).all()
            assert (s[[0, 2]] == scale).all()
        got.append([t[1].clone() for t in (kp, vp)] + [t[1].clone() for t in (ks, vs)])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a[:, :21] if a.dim() == 3 else a, b[:, :21] if b.dim() == 3 else b)
    pc.free()


def test_write8_scale_grows_by_far(wi):
    """A row 2^40 and 2^190 times as large as those in front of it, which become nothing; and back to small ones, which keep
    the large scale."""
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 1, 1, 1, rotary_dim=0))
    q = torch.ones((1, 1, 128), dtype=torch.bfloat16, device=DEV)
    pools = [(np.full((1, 1, 16, 128), 3.0), np.zeros((1, 1, 1), int))] * 2
    (kp, ks), (vp, vs) = (upload(p) for p in pools)
    expect = pools[0]
    for t, size in enumerate([1e-30, 1e-20, 1.0, 1e12, 3e38, 1.0, 1e37]):
        x, X = bf(np.linspace(-1, 1, 128).reshape(1, 1, 128) * size)
        pc.write8(q, x, x, i32([0]), i32([t]), kp, vp, ks, vs)
        expect = paged.append8(*expect, X, [t])
        for p, s in ((kp, ks), (vp, vs)):
            np.testing.assert_array_equal(exps8(s), expect[1])
            np.testing.assert_array_equal(values8(p), expect[0])
    pc.check()
    pc.free()


def test_write8_then_attention8_of_one_token_many_times(wi):
    """A decode loop on one stream with no waits between its calls: each step sees the token that it has just written."""
    rng = np.random.default_rng(65)
    hq, hkv, page, steps, n0 = 8, 2, 16, 40, 130
    n_pages = -(-(n0 + steps) // page)
    pools = [random_pool(rng, n_pages, hkv, page) for _ in range(2)]
    (kp, ks), (vp, vs) = (upload(p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 1, n_pages, rotary_dim=0))
    table = i32([range(n_pages)])
    x, X = bf(rng.normal(size=(steps, hq + 2 * hkv, 128)))
    outs = []
    for i in range(steps):
        q = pc.write8(x[i:i + 1, :hq], x[i:i + 1, hq:hq + hkv], x[i:i + 1, hq + hkv:], i32([n0 + i]), i32([n0 + i]), kp, vp, ks, vs)
        outs.append(pc.attention8(q, kp, vp, ks, vs, table, i32([0, 1]), i32([n0 + i + 1])))
    pc.check()
    pc.free()
    for i in range(steps):
        for w, part in enumerate((X[i:i + 1, hq:hq + hkv], X[i:i + 1, hq + hkv:])):
            pools[w] = paged.append8(*pools[w], part, [n0 + i])
        K, V = (paged.widened(*p) for p in pools)
        compare(f64(outs[i]), None, X[i:i + 1, :hq], K, V, [range(n_pages)], [0, 1], [n0 + i + 1])
    for p, s, r in ((kp, ks, pools[0]), (vp, vs, pools[1])):
        np.testing.assert_array_equal(exps8(s), r[1])
        np.testing.assert_array_equal(values8(p), r[0])


def test_outputs_of_another_alignment(wi):
    """out behind sixteen bytes of another buffer: the outputs are the same."""
    rng = np.random.default_rng(66)
    table, n_pages = lay_out([300], 16, rng)
    (k, ks), (v, vs) = (upload(random_pool(rng, n_pages, 2, 16)) for _ in range(2))
    pc = wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, 1, table.shape[1]))
    for n in (1, 40):
        q = bf(rng.normal(size=(n, 8, 128)))[0]
        args = (k, v, ks, vs, i32(table), i32([0, n]), i32([300]))
        a = pc.attention8(q, *args)
        buf = torch.zeros(n * 1024 + 16, dtype=torch.bfloat16, device=DEV)
        b, p = buf[8:8 + n * 1024].view(n, 8, 128), torch.empty(n * 1024 + 8, dtype=torch.bfloat16, device=DEV)[8:].view(n, 8, 128)
        p.copy_(q)
        pc.attention8(p, *args, out=b)
        pc.check()
        assert torch.equal(a, b) and (buf[:8] == 0).all() and (buf[8 + n * 1024:] == 0).all()
    pc.free()


@pytest.mark.parametrize("call", ["write8", "attention8", "gather8"])
def test_a_launch_that_fails_leaves_nothing_behind(wi, call):
    """A call on the default stream while a stream that waits for it is captured cannot be launched: it says so, and the
    next call is fine."""
    import ctypes

    cu = ctypes.CDLL("libcuda.so.1")
    pc = wi.PagedCache(wi.make_paged_config(4, 2, 16, 8, 1, 4))
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    q, kn = torch.zeros((1, 4, 128), **bf16), torch.zeros((1, 2, 128), **bf16)
    vn, qo, out = kn.clone(), q.clone(), q.clone()
    pools = [torch.zeros((8, 2, 16, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
    pools += [torch.zeros((8, 2, 1), dtype=torch.uint8, device=DEV) for _ in range(2)]
    rows = [torch.zeros((1, 1, 2, 4, 128), **bf16) for _ in range(2)]
    table, one, start = i32([[0, 1, 2, 3]]), [i32([1]) for _ in range(2)], i32([0, 1])
    run = {"write8": lambda s: pc.write8(q, kn, vn, one[0], one[1], *pools, qo, stream=s),
           "attention8": lambda s: pc.attention8(q, *pools, table, start, one[0], out=out, stream=s),
           "gather8": lambda s: pc.gather8(*pools, table, one[0], 0, *rows, stream=s)}[call]
    run(None)
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0
    assert cu.cuStreamBeginCapture_v2(stream, 0) == 0
    try:
        with pytest.raises(wi.WiError, match=f"paged {call} launch"):
            run(0)
    finally:
        cu.cuStreamEndCapture(stream, ctypes.byref(graph))     # the capture is lost with the refused call
        if graph.value:
            cu.cuGraphDestroy(graph)
        assert cu.cuStreamDestroy_v2(stream) == 0
    run(None)
    pc.check()
    pc.free()
