"""Calls of the paged cache in 8 bits that its documentation allows, on the GPU: layers of one allocation, queries in place, slots
that come twice, pages that requests share, axes that change.  What is compared here is the same call in a plainer form, bit
for bit, or the oracle with the tolerances that tests/test_gpu_paged8.py derives."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import DEV, bf, f64, freqs, i32, lay_out
from test_gpu_paged8 import compare, exps8, random_pool, upload, values8, write8_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wi():
    import clustered_sparse_kv_gb300 as m
    return m


def split(x, hq, hkv):
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def ones8(n):
    return torch.ones(n, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [4, 37, 800]), ([30, 1, 70], [0, 15, 411])])
@pytest.mark.parametrize("hkv,page,n_pages", [(1, 16, 101), (3, 48, 37), (2, 16, 101)])
def test_layers_of_one_allocation(wi, new, ctx, hkv, page, n_pages):
    """A layer's scales begin at any byte: n_pages * n_kv_heads * page_size / 16 need not be even."""
    rng = np.random.default_rng(71)
    layers, hq, total = 3, 2 * hkv, sum(new)
    kv = [c + n for c, n in zip(ctx, new)]
    table, used = lay_out(kv, page, rng)
    assert used <= n_pages
    at = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)])
    who = np.repeat(np.arange(len(new)), new)
    slots = i32(table[who, at // page] * page + at % page)
    start = np.concatenate([[0], np.cumsum(new)])
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, len(new), table.shape[1], inv_freq=freqs(128)))
    one = [upload(random_pool(rng, layers * n_pages, hkv, page)) for _ in range(2)]
    (kp, ks), (vp, vs) = ((v.view(layers, n_pages, hkv, page, 128), s.view(layers, n_pages, hkv, page // 16)) for v, s in one)
    for layer in range(layers):
        x, _ = bf(rng.normal(size=(total, hq + 2 * hkv, 128)))
        here = [t[layer] for t in (kp, vp, ks, vs)]
        own = [t.clone() for t in here]
        rest = [t.clone() for t in (kp, vp, ks, vs)]
        out = []
        for p in (here, own):
            q = pc.write8(*split(x, hq, hkv), i32(at), slots, *p, q_weight=ones8(128), k_weight=ones8(128))
            out.append((q, pc.attention8(q, *p, i32(table), i32(start), i32(kv))))
        pc.check()
        for a, b in zip(here, own):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        for a, b in zip(*out):
            assert torch.equal(a, b)
        for a, b in zip((kp, vp, ks, vs), rest):      # the other layers stand as they were
            keep = [i for i in range(layers) if i != layer]
            assert torch.equal(a.view(torch.uint8)[keep], b.view(torch.uint8)[keep])
        K, V = paged.widened(values8(here[0]), exps8(here[2])), paged.widened(values8(here[1]), exps8(here[3]))
        compare(f64(out[0][1]), None, f64(out[0][0]), K, V, table, start, kv)
    n = max(kv)
    ko, vo = (torch.full((len(new), layers, hkv, n, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pc.gather8(kp, vp, ks, vs, i32(table), i32(kv), 0, ko, vo)
    pc.check()
    np.testing.assert_array_equal(f64(ko), paged.gather(paged.widened(values8(kp), exps8(ks)), table, kv, 0, n))
    np.testing.assert_array_equal(f64(vo), paged.gather(paged.widened(values8(vp), exps8(vs)), table, kv, 0, n))
    pc.free()


def test_index_of_several_layers(wi):
    """An index over 8-bit pools of several layers is that of the rows that gather8 gives."""
    rng = np.random.default_rng(72)
    batch, layers, hkv, page, n = 2, 3, 1, 16, 1024
    table, n_pages = lay_out([n + 5, n + 40], page, rng)
    n_pages += n_pages % 2 == 0
    one = [upload(random_pool(rng, layers * n_pages, hkv, page)) for _ in range(2)]
    (kp, ks), (vp, vs) = ((v.view(layers, n_pages, hkv, page, 128), s.view(layers, n_pages, hkv, 1)) for v, s in one)
    pc = wi.PagedCache(wi.make_paged_config(4, hkv, page, n_pages, batch, table.shape[1]))
    kv = i32([n + 5, n + 40])
    rows = [torch.empty((batch, layers, hkv, n, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pc.gather8(kp, vp, ks, vs, i32(table), kv, 0, *rows)
    cfg = wi.make_config(batch, layers, 4, hkv, n, seg_len=1024, clusters_per_seg=64, iters=2)
    a = wi.WaveIndex.build_paged(cfg, pc, kp, vp, i32(table), kv, k_scales=ks, v_scales=vs)
    b = wi.WaveIndex.build(cfg, *rows)
    q, _ = bf(rng.normal(size=(batch, layers, 4, 128)))
    assert torch.equal(a.decode(q), b.decode(q))
    for x in (a, b, pc):
        x.free()


@pytest.mark.parametrize("n", [1, 40, 700, 5000])
def test_write8_with_queries_in_place(wi, n):
    rng = np.random.default_rng(73)
    hq, hkv, page = 8, 2, 64
    table, n_pages = lay_out([n], page, rng)
    at = np.arange(n)
    slots = i32(table[0, at // page] * page + at % page)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 1, table.shape[1], inv_freq=freqs(64), rotary_dim=64))
    x, _ = bf(rng.normal(size=(n, hq + 2 * hkv, 128)))
    q, k, v = (t.contiguous() for t in split(x, hq, hkv))
    pools = [upload(random_pool(rng, n_pages, hkv, page)) for _ in range(2)]
    args = (pools[0][0], pools[1][0], pools[0][1], pools[1][1])
    want = pc.write8(q, k, v, i32(at), slots, *args)
    assert pc.write8(q, k, v, i32(at), slots, *args, q_out=q) is q
    pc.check()
    assert torch.equal(q, want)
    pc.free()


@pytest.mark.parametrize("total,longest", [(40, 6), (330, 3), (330, 9), (1300, 7), (4700, 5), (4700, 40)])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (6, 3), (2, 1)])
def test_write8_short_and_long_runs_together(wi, total, longest, hq, hkv):
    """Runs of up to four tokens go another way than longer ones, also in one tile; a request's tokens may be cut anywhere by
    their groups."""
    rng = np.random.default_rng(total + longest)
    new = []
    while sum(new) < total:
        new.append(int(rng.integers(1, longest + 1)))
    axis = [i % 2 for i in range(32)] if hkv == 3 else None
    write8_case(wi, new, rng.integers(0, 50, len(new)).tolist(), hq, hkv, 16 if hkv == 1 else 48, rotary=64 if hkv == 3 else 128,
                interleaved=hkv == 1, norm=hkv != 1, axis=axis, seed=total, pad=2)


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
@pytest.mark.parametrize("off", [0, 1, 7, 11])
@pytest.mark.parametrize("interleaved", [False, True])
def test_write8_short_runs_are_the_longer_ones(wi, rows, off, interleaved):
    """A short run's rows and scale are, bit for bit, those of the same run with rows of zeros behind it: infinities, NaN,
    zeros and very different sizes among them, and rows in front that are rounded again."""
    rng = np.random.default_rng(78)
    hq, hkv, page, requests = 4, 4, 16, 12
    long = 5 if off + 5 <= 16 else 16 - off
    x, _ = bf(rng.normal(size=(requests, long, hq + 2 * hkv, 128)) * 2.0 ** rng.integers(-40, 40, (requests, 1, 1, 1)))
    x[:, rows:] = 0
    for b, odd in ((1, float("inf")), (2, -float("inf")), (3, float("nan")), (4, 0.0), (5, 2.0 ** -130), (6, 3e38)):
        x[b, rng.integers(rows), hq:, rng.integers(128)] = odd
    x[7] = float("nan")
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, requests, requests, 1, inv_freq=freqs(128), interleaved=interleaved))
    pools = [random_pool(rng, requests, hkv, page) for _ in range(2)]
    got = []
    for n in (rows, long):
        (k, ks), (v, vs) = (upload(p) for p in pools)
        at = (off + np.arange(n))[None].repeat(requests, 0)
        slots = at + 16 * np.arange(requests)[:, None]
        y = x[:, :n].reshape(-1, hq + 2 * hkv, 128).contiguous()
        pc.write8(*split(y, hq, hkv), i32(at.reshape(-1)), i32(slots.reshape(-1)), k, v, ks, vs, q_weight=ones8(128),
                  k_weight=ones8(128))
        pc.check()
        got.append([t.view(torch.uint8) for t in (k[:, :, :off + rows], v[:, :, :off + rows], ks, vs)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    pc.free()


@pytest.mark.parametrize("n", [40, 600, 6000])
def test_write8_unordered_slots_spoil_their_groups_alone(wi, n):
    """The same slot twice, and a run backwards: those groups are unspecified, all else is as without these tokens."""
    rng = np.random.default_rng(74)
    hq, hkv, page = 4, 2, 32
    table, n_pages = lay_out([n], page, rng)
    at = np.arange(n)
    slots = table[0, at // page] * page + at % page
    bad = slots.copy()
    bad[17] = bad[18]
    bad[n - 8:n - 4] = bad[n - 8:n - 4][::-1].copy()
    groups = {int(slots[17]) // 16, *(int(s) // 16 for s in slots[n - 8:n - 4])}
    gone = np.where(np.isin(slots // 16, list(groups)), -1, slots)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 1, table.shape[1], inv_freq=freqs(128)))
    x, _ = bf(rng.normal(size=(n, hq + 2 * hkv, 128)))
    start = [random_pool(rng, n_pages, hkv, page) for _ in range(2)]
    got = []
    for s in (bad, gone):
        (k, ks), (v, vs) = (upload(p) for p in start)
        q = pc.write8(*split(x, hq, hkv), i32(at), i32(s), k, v, ks, vs)
        pc.check()
        got.append((q, k, v, ks, vs))
    assert torch.equal(got[0][0], got[1][0])
    keep = np.ones(n_pages * page // 16, bool)
    keep[list(groups)] = False
    for i in range(1, 5):
        a, b = (g[i].view(torch.uint8).cpu().numpy().reshape(n_pages, hkv, page // 16, -1) for g in got)
        a, b = (t.transpose(0, 2, 1, 3).reshape(n_pages * (page // 16), -1)[keep] for t in (a, b))
        np.testing.assert_array_equal(a, b)
    pc.free()


@pytest.mark.parametrize("new", [[1, 1, 1], [33, 200, 1]])
def test_requests_that_share_pages(wi, new):
    rng = np.random.default_rng(75)
    hq, hkv, page, shared = 8, 2, 16, 40
    kv = [shared * page + 3 + n for n in new]
    table, n_pages = lay_out(kv, page, rng)
    table[:, :shared] = table[0, :shared]
    start = np.concatenate([[0], np.cumsum(new)])
    pools = [random_pool(rng, n_pages, hkv, page) for _ in range(2)]
    (k, ks), (v, vs) = (upload(p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 3, table.shape[1]))
    q, Q = bf(rng.normal(size=(sum(new), hq, 128)))
    lse = torch.empty((sum(new), hq), device=DEV)
    out = pc.attention8(q, k, v, ks, vs, i32(table), i32(start), i32(kv), lse=lse)
    pc.check()
    compare(f64(out), f64(lse), Q, *(paged.widened(*p) for p in pools), table, start, kv)
    pc.free()


@pytest.mark.parametrize("batch,where,new,kv", [
    (30, range(30), 1, (300, 700)), (2, range(2), 1, (1, 2)), (38, range(38), 1, (900, 1100)),      # an item to a CTA
    (300, (3, 77, 78, 299), 1, (500, 520)), (4000, (0, 1999, 3999), 1, (100, 4000)),                # few of many requests
    (300, (3, 77, 78, 299), 5, (500, 520)), (16, range(16), 4, (1900, 2100)), (4000, (5, 3999), 90, (90, 700)),
    (20, range(20), 16, (16, 16)), (6, range(6), 33, (30, 800)), (3, range(3), 200, (200, 300))])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (7, 1), (8, 8)])
def test_requests_whole_in_their_ctas(wi, batch, where, new, kv, hq, hkv):
    """Batches with fewer items than CTAs, of lengths alike or not; requests without tokens between them; twice the same."""
    rng = np.random.default_rng(batch + new)
    page, counts = 16, np.zeros(batch, int)
    counts[list(where)] = new
    lengths = np.where(counts > 0, rng.integers(kv[0], kv[1] + 1, batch), rng.integers(0, 40, batch))
    table, n_pages = lay_out(lengths.tolist(), page, rng)
    start = np.concatenate([[0], np.cumsum(counts)])
    pools = [random_pool(rng, n_pages, hkv, page) for _ in range(2)]
    (k, ks), (v, vs) = (upload(p) for p in pools)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, batch, table.shape[1]))
    q, Q = bf(rng.normal(size=(int(start[-1]), hq, 128)))
    lse = torch.empty((len(q), hq), device=DEV)
    args = (q, k, v, ks, vs, i32(table), i32(start), i32(lengths))
    out = pc.attention8(*args, lse=lse)
    again = pc.attention8(*args)
    pc.check()
    assert torch.equal(out, again)
    compare(f64(out), f64(lse), Q, *(paged.widened(*p) for p in pools), table, start, lengths)
    pc.free()


def test_no_tokens_and_no_rows(wi):
    pc = wi.PagedCache(wi.make_paged_config(4, 2, 16, 4, 2, 2, inv_freq=freqs(128)), axes=[i % 3 for i in range(64)])
    rng = np.random.default_rng(76)
    (k, ks), (v, vs) = (upload(random_pool(rng, 4, 2, 16)) for _ in range(2))
    was = [t.clone() for t in (k, v, ks, vs)]
    none = torch.empty((0, 8, 128), dtype=torch.bfloat16, device=DEV)
    q = pc.write8(*split(none, 4, 2), torch.empty((3, 0), dtype=torch.int32, device=DEV), i32([]), k, v, ks, vs)
    assert q.shape == (0, 4, 128)
    assert pc.attention8(q, k, v, ks, vs, i32([[0, 1], [2, 3]]), i32([0, 0, 0]), i32([5, 20])).shape == (0, 4, 128)
    out = torch.empty((1, 1, 2, 0, 128), dtype=torch.bfloat16, device=DEV)
    pc.gather8(k, v, ks, vs, i32([[0, 1]]), i32([5]), 32, out, out.clone())
    pc.check()
    for a, b in zip((k, v, ks, vs), was):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    pc.free()


def test_captured_writes_keep_their_axes(wi):
    """A graph goes on with the axes that it was captured with; a later call has the handle's."""
    rng = np.random.default_rng(77)
    hq, hkv, page, n, n_pages = 4, 2, 16, 50, 4
    axes = [i % 3 for i in range(64)]
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 1, n_pages, inv_freq=freqs(128)), axes=axes)
    plain = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 1, n_pages, inv_freq=freqs(128)))
    x, _ = bf(rng.normal(size=(n, hq + 2 * hkv, 128)))
    pos, slots = i32(rng.integers(0, 900, (3, n))), i32(np.arange(n))

    def pools():
        return [torch.zeros((n_pages, hkv, page, 128), dtype=torch.uint8, device=DEV) for _ in range(2)] + \
               [torch.zeros((n_pages, hkv, 1), dtype=torch.uint8, device=DEV) for _ in range(2)]

    eager, mine, after, single = pools(), pools(), pools(), pools()
    q0 = pc.write8(*split(x, hq, hkv), pos, slots, *eager)
    q1 = torch.zeros_like(q0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pc.write8(*split(x, hq, hkv), pos, slots, *mine, q1)
    side.synchronize()
    for t in (*mine, q1):
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pc.write8(*split(x, hq, hkv), pos, slots, *mine, q1)
    assert wi.lib.wi_paged_axes(pc.handle, 1, None) == 0
    g.replay()
    # the C call now reads [1][n] positions
    q2 = torch.zeros_like(q0)
    q, k, v = split(x, hq, hkv)
    step = (hq + 2 * hkv) * 128
    rc = wi.lib.wi_paged_write8(pc.handle, n, q.data_ptr(), step, k.data_ptr(), step, v.data_ptr(), step, None, None,
                                pos.data_ptr(), slots.data_ptr(), q2.data_ptr(), *(t.data_ptr() for t in after),
                                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    q3 = plain.write8(q, k, v, pos[0], slots, *single)
    pc.check(), plain.check()
    for a, b in zip((*eager, q0, *after, q2), (*mine, q1, *single, q3)):
        assert torch.equal(a, b)
    assert not torch.equal(q0, q2)
    pc.free(), plain.free()
