"""The paged cache on the GPU against oracle.paged (float64), on the same input bytes.

Tolerances.  A bf16 output is off by at most half a step, 2^-8 of its value.  On top of that:
  write: the fp32 terms of a rotated pair are each exact to a few 2^-24 (products, rsqrt and sincospi of 2 ulp, the
    angle of 2^-32 turns), at most 2^-19 of |a| + |b| in all;
  attention: weights rounded to bf16, 2^-8 of sum w|v|; a score is an fp32 dot of 128 products, off by at most
    128 * 2^-24 of sum |q k| / sqrt(128) (and its weight by that much, relatively, through the exponential, once
    itself and once through the sum of the weights); the sums over n positions in fp32, n * 2^-24 each;
  lse: the score's error, and n * 2^-24 of the sum.
Integers and copies are equal.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import paged

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
THETA = 500000.0


@pytest.fixture(scope="module")
def wi():
    import clustered_sparse_kv_gb300 as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bf(x):
    """bf16 tensor on the device and its float64 values."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(DEV).bfloat16()
    return t, t.double().cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def lay_out(kv, page, rng, spare=3):
    """A block table for requests of these lengths with pages in random order, and the pool's page count."""
    used = [-(-max(n, 0) // page) for n in kv]
    n_pages = sum(used) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(kv), max(used + [1])), -1, np.int64)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def freqs(rotary):
    return [THETA ** (-2.0 * i / rotary) for i in range(rotary // 2)]


# ------------------------------------------------------------------ tables ----

def run_tables(pc, ctx, new, free, n_free, table, n_tokens, fill=-7):
    a = {"block_table": i32(table), "kv_len": i32([fill] * len(ctx)), "q_start": i32([fill] * (len(ctx) + 1)),
         "slots": i32([fill] * n_tokens), "positions": i32([fill] * n_tokens), "n_free_out": i32([fill])}
    pc.tables(i32(ctx), i32(new), i32(free), i32([n_free]), **a)
    return {k: v.cpu().numpy().astype(np.int64) for k, v in a.items()}


@pytest.mark.parametrize("batch,page,ctx_hi,new_hi,pad", [
    (1, 16, 0, 1, 0), (1, 16, 40, 1, 1), (3, 16, 100, 50, 5), (8, 48, 1000, 3, 0), (64, 64, 500, 200, 100),
    (255, 16, 64, 33, 0), (257, 128, 3000, 40, 7), (1000, 16, 50, 2, 600), (4096, 32, 70, 3, 11), (2, 16, 10, 40000, 3),
])
def test_tables(wi, batch, page, ctx_hi, new_hi, pad):
    rng = np.random.default_rng(batch)
    ctx, new = rng.integers(0, ctx_hi + 1, batch), rng.integers(0, new_hi + 1, batch)
    new[rng.integers(0, batch)] = new_hi
    held, n_pages = lay_out(ctx, page, rng, spare=0)
    width = int(max(-(-(ctx + new) // page))) + 1
    fresh = int((-(-(ctx + new) // page) - -(-ctx // page)).sum())
    table = np.full((batch, width), -5)
    table[:, :held.shape[1]] = np.where(held[:, :width] >= 0, held[:, :width], -5)
    free = n_pages + rng.permutation(fresh + 4)
    pc = wi.PagedCache(wi.make_paged_config(1, 1, page, n_pages + fresh + 4, batch, width))
    n_tokens = int(new.sum()) + pad
    for n_free in (fresh + 4, fresh):   # some left, none left
        got = run_tables(pc, ctx, new, free, n_free, table, n_tokens)
        ref = paged.page_tables(ctx, new, free, n_free, table, page, n_tokens)
        for k in ref:
            np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
        again = run_tables(pc, ctx, new, free, n_free, got["block_table"], n_tokens)  # idempotent
        for k in ref:
            np.testing.assert_array_equal(again[k], ref[k], err_msg=k)
    pc.check()
    pc.free()


@pytest.mark.parametrize("what", ["pages", "tokens", "negative new", "negative ctx", "too long", "n_free", "overflow"])
def test_tables_refuse_a_step_as_a_whole(wi, what):
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 40, 4, 8))
    ctx, new, n_free, n_tokens = [20, 0, 33], [5, 40, 1], 10, 50
    if what == "pages":
        n_free = 3                      # one request needs three, another none, the last none: 3 + 0; make it four
        new[2] = 17
    if what == "tokens":
        n_tokens = 45
    if what == "negative new":
        new[1] = -1
    if what == "negative ctx":
        ctx[1] = -3
    if what == "too long":
        new[0] = 109
    if what == "n_free":
        n_free = 21
    if what == "overflow":
        ctx, new = [0, 2 ** 31 - 1, 5], [2 ** 31 - 1] * 3
    table = np.full((3, 8), 2)
    got = run_tables(pc, ctx, new, list(range(20)), n_free, table, n_tokens)
    np.testing.assert_array_equal(got["block_table"], table)
    assert (got["slots"] == -1).all() and (got["positions"] == -1).all() and (got["q_start"] == 0).all()
    np.testing.assert_array_equal(got["kv_len"], [c if 0 <= c <= 128 else 0 for c in ctx])
    assert got["n_free_out"][0] == n_free
    with pytest.raises(wi.WiError, match="more pages" if what == "pages" else "length"):
        pc.check()
    pc.check()   # reported once
    pc.free()


def test_tables_report_bad_pages_and_give_no_slot(wi):
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 6, 2, 4))
    got = run_tables(pc, [17, 15], [2, 2], [6, 5], 2, [[0, -1, -1, -1], [1, -1, -1, -1]], 4)
    # request 0 continues in its second page, which its row does not have; request 1 opens a page: the last
    # free one, 5, is fine
    assert got["slots"].tolist() == [-1, -1, 31, 80]
    with pytest.raises(wi.WiError, match="page or slot"):
        pc.check()
    got = run_tables(pc, [16, 0], [1, 1], [5, 6], 2, [[0, -1, -1, -1], [-1, -1, -1, -1]], 2)   # page 6 of 6
    assert got["slots"].tolist() == [-1, 80]
    with pytest.raises(wi.WiError, match="page or slot"):
        pc.check()
    pc.free()


# ------------------------------------------------------------------ write ----

def write_case(wi, n, hq, hkv, page, rotary, interleaved, norm, seed, layout="fused", far=1 << 20, scale=1.0, pad=0):
    rng = np.random.default_rng(seed)
    total = n + pad
    fused, F = bf(rng.normal(size=(total, hq + 2 * hkv, 128)) * rng.choice([0.01, 1, 30], size=(total, 1, 1)))
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    if layout == "separate":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    Q, K, V = F[:, :hq], F[:, hq:hq + hkv], F[:, hq + hkv:]
    n_pages = -(-n // page) + 2
    slots = rng.permutation(n_pages * page)[:total]
    pos = rng.integers(0, far, total)
    pos[:min(n, 2)] = [0, far - 1][:min(n, 2)]
    pos[n:] = -1
    if n > 4:
        slots[3] = -1            # its query is wanted, its key and value are not
    wq, WQ = bf(1 + rng.normal(size=128) * 0.3)
    wk, WK = bf(1 + rng.normal(size=128) * 0.3)
    f = freqs(rotary)
    eps = 1e-5
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 1, 1, rotary_dim=rotary, interleaved=interleaved,
                                            inv_freq=f, eps=eps, rope_scale=scale))
    kp = torch.full((n_pages, hkv, page, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    out = torch.full((total, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    pc.write(q, k, v, i32(pos), i32(slots), kp, vp, out, wq if norm else None, wk if norm else None)
    pc.check()
    rq, nq = paged.norm_rotate(Q[:n], WQ if norm else None, eps, pos[:n], f, interleaved, scale)
    rk, nk = paged.norm_rotate(K[:n], WK if norm else None, eps, pos[:n], f, interleaved, scale)

    def near(got, ref, normed):
        size = np.abs(normed)
        h = rotary // 2
        if rotary:   # |a| + |b| of the pair
            a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, h), slice(h, rotary))
            both = (size[..., a] + size[..., b]) * max(abs(scale), 1)
            size[..., a] = size[..., b] = both
        err = np.abs(got - ref)
        tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * 2.0 ** -19 * size + 2.0 ** -133
        assert (err <= tol).all(), (err / tol).max()

    got = f64(out)
    near(got[:n], rq, nq)
    assert (got[n:] == 7).all()
    GK, GV = (f64(x).transpose(0, 2, 1, 3).reshape(-1, hkv, 128) for x in (kp, vp))
    stored = np.nonzero((slots >= 0) & (pos >= 0))[0]
    near(GK[slots[stored]], rk[stored], nk[stored])
    np.testing.assert_array_equal(GV[slots[stored]], V[stored])
    rest = np.setdiff1d(np.arange(n_pages * page), slots[stored])
    assert (GK[rest] == 7).all() and (GV[rest] == 7).all()
    pc.free()


@pytest.mark.parametrize("rotary,interleaved", [(128, False), (128, True), (64, False), (64, True), (8, False),
                                                (8, True), (96, False), (120, True), (0, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_write_rotations(wi, rotary, interleaved, norm):
    write_case(wi, 37, 6, 2, 16, rotary, interleaved, norm, seed=rotary + norm, pad=3)


@pytest.mark.parametrize("n,hq,hkv,page", [(1, 32, 8, 16), (1, 1, 1, 16), (2, 28, 4, 48), (17, 5, 5, 16), (130, 8, 1, 64),
                                           (300, 7, 1, 256)])
@pytest.mark.parametrize("layout", ["fused", "separate"])
def test_write_sizes(wi, n, hq, hkv, page, layout):
    write_case(wi, n, hq, hkv, page, 128, False, True, seed=n + hq, layout=layout)


def test_write_far_positions_and_scale(wi):
    write_case(wi, 40, 4, 1, 16, 128, False, True, seed=5, far=2 ** 31 - 1, scale=1.25)
    write_case(wi, 40, 4, 1, 16, 64, True, False, seed=6, far=2 ** 31 - 1, scale=0.5)


def test_write_many_tokens_take_every_head_in_one_go(wi):
    """More tokens than the launch has room to spread: the same rows as in small calls, bit for bit."""
    rng = np.random.default_rng(9)
    n, hq, hkv = 6001, 28, 4
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, 16, 400, 1, 1))
    x = torch.from_numpy(rng.normal(size=(n, (hq + 2 * hkv) * 128)).astype(np.float32)).to(DEV).bfloat16()
    q, k, v = x.split([hq * 128, hkv * 128, hkv * 128], 1)
    q, k, v = q.view(n, hq, 128), k.view(n, hkv, 128), v.view(n, hkv, 128)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    slots, pos = i32(rng.permutation(6400)[:n]), i32(rng.integers(0, 10 ** 6, n))
    whole = [torch.zeros((400, hkv, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    a = pc.write(q, k, v, pos, slots, whole[0], whole[1], None, w, w)
    b = torch.empty_like(a)
    for i in range(0, n, 50):
        s = slice(i, min(i + 50, n))
        pc.write(q[s], k[s], v[s], pos[s], slots[s], whole[2], whole[3], b[s], w, w)
    pc.check()
    assert torch.equal(a, b) and torch.equal(whole[0], whole[2]) and torch.equal(whole[1], whole[3])
    pc.free()


def test_write_in_place_and_without_slots(wi):
    rng = np.random.default_rng(11)
    n, hq, hkv = 9, 4, 2
    f = freqs(128)
    q, Q = bf(rng.normal(size=(n, hq, 128)))
    k, K = bf(rng.normal(size=(n, hkv, 128)))
    v, V = bf(rng.normal(size=(n, hkv, 128)))
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, 16, 4, 1, 1, inv_freq=f))
    pos = rng.integers(0, 10 ** 6, n)
    want = pc.write(q, k, v, i32(pos), i32(np.arange(n)), *(torch.zeros((4, hkv, 16, 128), dtype=torch.bfloat16,
                                                                        device=DEV) for _ in range(2)))
    kn, vn = torch.zeros_like(k), torch.zeros_like(v)
    got = pc.write(q, k, v, i32(pos), None, kn, vn, q_out=q)
    pc.check()
    assert got is q and torch.equal(q, want) and torch.equal(vn, v)
    rk, nk = paged.norm_rotate(K, None, 1, pos, f)
    pair = np.abs(nk[..., :64]) + np.abs(nk[..., 64:])
    tol = 2.0 ** -8 * np.abs(rk) + 2.0 ** -18 * np.concatenate([pair, pair], -1)
    assert (np.abs(f64(kn) - rk) <= tol).all()
    pc.free()


def test_write_zero_rows_and_bad_slots(wi):
    pc = wi.PagedCache(wi.make_paged_config(2, 1, 16, 2, 1, 1))
    z = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    kp = torch.full((2, 1, 16, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    out = pc.write(z[:, :2], z[:, 2:3], z[:, 3:], i32([0, 1, 2]), i32([0, 31, 32]), kp, vp, None, w, w)
    assert (out == 0).all()       # a zero vector stays zero under the norm
    assert (kp.view(-1, 128)[[0, 31]] == 0).all() and (kp.view(-1, 128)[1:31] == 3).all()
    with pytest.raises(wi.WiError, match="page or slot"):   # slot 32 of 32
        pc.check()
    pc.free()


# ------------------------------------------------------------------ attention ----

def attention_case(wi, hq, hkv, page, new, kv, seed, pad=0, scale=1.0, poison=None, want_lse=True):
    rng = np.random.default_rng(seed)
    table, n_pages = lay_out(kv, page, rng)
    q_start = np.concatenate([[0], np.cumsum(new)])
    n = int(q_start[-1]) + pad
    q, Q = bf(rng.normal(size=(max(n, 1), hq, 128)) * scale)
    Kp, Vp = (rng.normal(size=(n_pages, hkv, page, 128)) + rng.normal(size=(hkv, 1, 128)) for _ in range(2))
    if poison is not None:
        poison(Kp, Vp, table)
    k, K = bf(Kp)
    v, V = bf(Vp)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, len(kv), table.shape[1]))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV) if want_lse else None
    args = (q, k, v, i32(table), i32(q_start), i32(kv))
    pc.attention(*args, out=out, lse=lse)
    pc.check()
    live = slice(0, int(q_start[-1]))
    ref, rlse, spread = paged.attention(Q, K, V, table, q_start, kv)
    got = f64(out)
    assert (got[q_start[-1]:] == 7).all()
    # the largest sum |q k| / sqrt(128) of a row is at most |q| max|k| / sqrt(128)
    finite = np.where(np.isfinite(K), K, 0)
    top = np.linalg.norm(Q[live], axis=-1) * np.sqrt((finite ** 2).sum(-1).max()) / np.sqrt(128)
    ds = 128 * 2.0 ** -24 * top + 2.0 ** -20
    most = max([1, *kv])
    tol = (2.0 ** -8 * np.abs(ref[live]) +
           (1 + 2.0 ** -7) * spread[live] * (2.0 ** -8 + 2 * ds + 2 * most * 2.0 ** -24)[..., None] + 2.0 ** -133)
    good = np.isfinite(ref[live])
    err = np.abs(np.where(good, got[live], 0) - np.where(good, ref[live], 0))
    if err.size:
        assert (err[good] <= tol[good]).all(), (err[good] / tol[good]).max()
        np.testing.assert_array_equal(got[live][~good], ref[live][~good])
    if want_lse:
        gl = lse.double().cpu().numpy()
        assert (gl[q_start[-1]:] == 7).all()
        same = gl[live] == rlse[live]     # -infinity where a row sees nothing
        ltol = ds + most * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(rlse[live]), rlse[live], 0)) + 2.0 ** -20
        with np.errstate(invalid="ignore"):
            assert (same | (np.abs(gl[live] - rlse[live]) <= ltol)).all()
    again = torch.full_like(out, 7.0)
    pc.attention(*args, out=again)        # same bits, with and without lse
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    pc.check()
    pc.free()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 1), (10, 2), (6, 1), (28, 4), (8, 1), (32, 8)])
@pytest.mark.parametrize("new,ctx", [(1, 200), (5, 0), (19, 300), (70, 61)])
def test_attention_heads(wi, hq, hkv, new, ctx):
    attention_case(wi, hq, hkv, 16, [new], [ctx + new], seed=hq + new)


@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 383, 1000, 4097])
@pytest.mark.parametrize("page", [16, 48, 128, 8192])
def test_attention_single_token_lengths(wi, kv, page):
    attention_case(wi, 8, 2, page, [1], [kv], seed=kv)


@pytest.mark.parametrize("new", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 260, 700])
@pytest.mark.parametrize("ctx", [0, 1, 100, 128, 515])
def test_attention_chunk_lengths(wi, new, ctx):
    attention_case(wi, 4, 1, 64, [new], [ctx + new], seed=new + ctx)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 96, 112, 128, 256, 1024, 1040])
def test_attention_page_sizes(wi, page):
    attention_case(wi, 4, 2, page, [40, 1, 130], [700, 333, 131], seed=page)


@pytest.mark.parametrize("seed", range(8))
def test_attention_mixed_requests(wi, seed):
    rng = np.random.default_rng(100 + seed)
    hq, hkv = [(28, 4), (8, 2), (6, 1), (16, 8), (5, 1), (4, 4), (32, 8), (3, 3)][seed]
    batch = int(rng.integers(2, 30))
    new = rng.choice([0, 1, 1, 1, 2, 7, 40, 150], size=batch)
    ctx = rng.choice([0, 0, 3, 16, 127, 500, 1300, 2000], size=batch)
    attention_case(wi, hq, hkv, int(rng.choice([16, 48, 64])), list(new), list(ctx + new), seed, pad=int(seed % 3))


def test_attention_long_single_tokens(wi):
    attention_case(wi, 8, 2, 16, [1, 1, 1], [30001, 5, 12000], seed=1)


def test_attention_many_short_requests(wi):
    rng = np.random.default_rng(3)
    kv = rng.integers(1, 40, 700)
    attention_case(wi, 4, 2, 16, [1] * 700, list(kv), seed=2)


def test_attention_large_scores(wi):
    """Scores of a few hundred: the running maximum moves far, and most weights are zero."""
    attention_case(wi, 4, 2, 16, [90, 1], [600, 900], seed=4, scale=30.0)


def test_attention_rows_that_see_nothing(wi):
    # fewer cached positions than new tokens: the first tokens sit before position 0
    attention_case(wi, 4, 1, 16, [10, 300, 1, 200], [3, 100, 0, 0], seed=5)
    attention_case(wi, 28, 4, 16, [1, 1, 40], [0, 1, 39], seed=6)


def test_attention_no_tokens(wi):
    attention_case(wi, 4, 1, 16, [0, 0], [50, 0], seed=7, pad=4)


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf, 3e38])
@pytest.mark.parametrize("new,ctx", [([1], [20]), ([40], [0]), ([150, 1, 9], [90, 300, 119]), ([300], [1])])
def test_attention_poison_behind_the_last_position(wi, value, new, ctx):
    kv = [n + c for n, c in zip(new, ctx)]

    def poison(K, V, table):
        for b, n in enumerate(kv):
            j, r = divmod(n, K.shape[2])
            if r:
                K[table[b, j], :, r:] = value
                V[table[b, j], :, r:] = value
        held = table[table >= 0]
        other = np.setdiff1d(np.arange(len(K)), held)
        K[other] = value
        V[other] = value

    attention_case(wi, 8, 2, 16, new, kv, seed=8, poison=poison)
    attention_case(wi, 8, 2, 128, new, kv, seed=8, poison=poison)


@pytest.mark.parametrize("hq,hkv", [(4, 1), (7, 1), (1, 1)])
@pytest.mark.parametrize("at", [130, 200, 259])
def test_attention_poison_at_later_positions(wi, hq, hkv, at):
    """Infinities and NaN of a later token reach the tokens that see it and no others."""
    def poison(K, V, table):
        page = K.shape[2]
        K[table[0, at // page], :, at % page, 5] = np.nan
        V[table[0, at // page], :, at % page, 9] = np.nan
        V[table[0, at // page], :, at % page, 70] = np.nan

    rng = np.random.default_rng(9)
    new, kv = [160, 1], [260, 50]
    table, n_pages = lay_out(kv, 16, rng)
    q, Q = bf(rng.normal(size=(161, hq, 128)))
    Kp, Vp = (rng.normal(size=(n_pages, hkv, 16, 128)) for _ in range(2))
    clean = [bf(x)[0] for x in (Kp, Vp)]
    poison(Kp, Vp, table)
    dirty = [bf(x)[0] for x in (Kp, Vp)]
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, 16, n_pages, 2, table.shape[1]))
    args = (i32(table), i32([0, 160, 161]), i32(kv))
    a, b = pc.attention(q, *clean, *args), pc.attention(q, *dirty, *args)
    pc.check()
    sees = at - 100
    assert torch.equal(a[:sees], b[:sees]) and torch.equal(a[160], b[160])
    assert b[sees:160].isnan().all()      # through the score, every element
    pc.free()


@pytest.mark.parametrize("at", [30, 128, 141, 259])
def test_attention_poison_in_a_value_alone(wi, at):
    """One infinite and one NaN element of a token's value: in the rows that see it those two elements and no
    others, in the rest nothing."""
    def poison(K, V, table):
        page = K.shape[2]
        V[table[0, at // page], :, at % page, 9] = np.inf
        V[table[0, at // page], :, at % page, 70] = np.nan

    attention_case(wi, 4, 1, 16, [260], [260], seed=10, poison=poison)
    attention_case(wi, 7, 1, 64, [200, 1], [260, 70], seed=10, poison=poison)


def test_attention_reports_bad_tables(wi):
    rng = np.random.default_rng(12)
    pc = wi.PagedCache(wi.make_paged_config(4, 1, 16, 8, 2, 4))
    q, _ = bf(rng.normal(size=(3, 4, 128)))
    k, _ = bf(rng.normal(size=(8, 1, 16, 128)))
    v, _ = bf(rng.normal(size=(8, 1, 16, 128)))
    good = [[1, 2, 3, -1], [4, 5, -1, -1]]
    ref = pc.attention(q, k, v, i32(good), i32([0, 2, 3]), i32([40, 20]))
    pc.check()
    for table, start, kv, match, intact in [
            ([[1, 8, 3, -1], [4, 5, -1, -1]], [0, 2, 3], [40, 20], "page or slot", [2]),
            ([[1, 2, 3, -1], [4, -1, -1, -1]], [0, 2, 3], [40, 20], "page or slot", [0, 1]),
            (good, [0, 2, 3], [40, 65], "length", [0, 1]),
            (good, [0, 2, 3], [-1, 20], "length", [2]),
            (good, [0, 2, 4], [40, 20], "length", [0, 1]),
            (good, [0, 2, 1], [40, 20], "length", [0, 1])]:
        out = torch.full_like(q, 7.0)
        pc.attention(q, k, v, i32(table), i32(start), i32(kv), out=out)
        with pytest.raises(wi.WiError, match=match):
            pc.check()
        assert torch.equal(out[intact], ref[intact]), (table, start, kv)
    pc.check()
    pc.free()


def test_attention_beyond_32_bit_offsets(wi):
    """A pool of more than 2^32 elements; a request whose pages lie at both ends."""
    hkv, page, n_pages = 2, 64, 270000      # 270000 * 2 * 64 * 128 elements: 8.8 GB each
    k = torch.empty((n_pages, hkv, page, 128), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    rng = np.random.default_rng(13)
    table = np.array([[n_pages - 1, 0, n_pages - 2, 131072]])
    K, V = (rng.normal(size=(4, hkv, page, 128)) for _ in range(2))
    for i, p in enumerate(table[0]):
        k[p], K[i] = bf(K[i])
        v[p], V[i] = bf(V[i])
    q, Q = bf(rng.normal(size=(30, 4, 128)))
    pc = wi.PagedCache(wi.make_paged_config(4, hkv, page, n_pages, 1, 4))
    out = pc.attention(q, k, v, i32(table), i32([0, 30]), i32([250]))
    ko, vo = (torch.empty((1, 1, hkv, 100, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pc.gather(k, v, i32(table), i32([250]), 120, ko, vo)
    slots = [int(table[0, p // page]) * page + p % page for p in (0, 140, 200)]
    kv = torch.ones((3, hkv, 128), dtype=torch.bfloat16, device=DEV)
    pc.check()
    ref, _, spread = paged.attention(Q, K, V, [[0, 1, 2, 3]], [0, 30], [250])
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread).all()
    np.testing.assert_array_equal(f64(ko), paged.gather(K[None], [[0, 1, 2, 3]], [250], 120, 100))
    np.testing.assert_array_equal(f64(vo), paged.gather(V[None], [[0, 1, 2, 3]], [250], 120, 100))
    pc.write(q[:3], kv, kv * 2, i32([0, 0, 0]), i32(slots), k, v)
    pc.check()
    for s in slots:
        assert (k[s // page, :, s % page] == 1).all() and (v[s // page, :, s % page] == 2).all()
    pc.free()


# ------------------------------------------------------------------ gather ----

@pytest.mark.parametrize("batch,layers,hkv,page,pos0,n,kv_hi", [
    (1, 1, 1, 16, 0, 1, 1), (1, 1, 8, 16, 0, 300, 300), (3, 2, 2, 48, 17, 100, 160), (16, 3, 4, 16, 40, 1, 60),
    (2, 1, 3, 64, 0, 513, 400), (5, 2, 1, 1024, 999, 65, 2000), (1, 1, 2, 16, 200, 50, 100)])
def test_gather(wi, batch, layers, hkv, page, pos0, n, kv_hi):
    rng = np.random.default_rng(batch + n)
    kv = rng.integers(0, kv_hi + 1, batch)
    kv[0] = kv_hi
    table, n_pages = lay_out(kv, page, rng)
    width = max(table.shape[1], -(-(pos0 + n) // page))
    table = np.concatenate([table, np.full((batch, width - table.shape[1]), -1)], 1)
    k, K = bf(rng.normal(size=(layers, n_pages, hkv, page, 128)))
    v, V = bf(rng.normal(size=(layers, n_pages, hkv, page, 128)))
    pc = wi.PagedCache(wi.make_paged_config(hkv, hkv, page, n_pages, batch, width))
    ko, vo = (torch.full((batch, layers, hkv, n, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pc.gather(k if layers > 1 else k[0], v if layers > 1 else v[0], i32(table), i32(kv), pos0, ko, vo)
    pc.check()
    np.testing.assert_array_equal(f64(ko), paged.gather(K, table, kv, pos0, n))
    np.testing.assert_array_equal(f64(vo), paged.gather(V, table, kv, pos0, n))
    pc.free()


def test_gather_reports_bad_tables(wi):
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 4, 2, 4))
    k = torch.ones((4, 1, 16, 128), dtype=torch.bfloat16, device=DEV)
    ko, vo = (torch.full((2, 1, 1, 20, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for table, kv, match in [([[0, 4, -1, -1], [1, 2, -1, -1]], [20, 20], "page or slot"),
                             ([[0, 3, -1, -1], [1, 2, -1, -1]], [65, 20], "length")]:
        pc.gather(k, k.clone(), i32(table), i32(kv), 0, ko, vo)
        with pytest.raises(wi.WiError, match=match):
            pc.check()
        assert (ko[1] == 1).all()
    pc.free()


# ------------------------------------------------------- refusals of the calls ----

def test_calls_refuse_bad_arguments(wi):
    pc = wi.PagedCache(wi.make_paged_config(4, 2, 16, 8, 2, 4))
    P = lambda t: t.data_ptr()  # noqa: E731
    i = [i32([0, 0, 0, 0, 0]) for _ in range(10)]
    x = torch.zeros((4, 6, 128), dtype=torch.bfloat16, device=DEV)
    o = [torch.zeros((8, 2, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    lib, h = wi.lib, pc.handle

    def tables(batch=1, n=1, cap=1, **kw):
        names = ["ctx", "new", "free", "nfree", "table", "kv", "start", "slots", "pos", "out"]
        p = {k: P(t) for k, t in zip(names, i)}
        p.update(kw)
        return lib.wi_paged_tables(h, batch, p["ctx"], p["new"], p["free"], p["nfree"], cap, p["table"], p["kv"],
                                   p["start"], p["slots"], p["pos"], n, p["out"], None)

    assert tables() == 0
    for kw in (dict(batch=0), dict(batch=3), dict(n=-1), dict(cap=-1), dict(ctx=None), dict(free=None), dict(slots=None),
               dict(kv=P(i[0])), dict(out=P(i[3])), dict(slots=P(i[8])), dict(pos=P(i[8]) + 2)):
        assert tables(**kw) == -1, kw

    def write(n=2, qs=768, ks=768, vs=768, **kw):
        p = dict(q=P(x), k=P(x) + 1024, v=P(x) + 1536, wq=None, wk=None, pos=P(i[0]), slots=P(i[1]), qo=P(o[0]),
                 kp=P(o[1]), vp=P(o[2]))
        p.update(kw)
        return lib.wi_paged_write(h, n, p["q"], qs, p["k"], ks, p["v"], vs, p["wq"], p["wk"], p["pos"], p["slots"],
                                  p["qo"], p["kp"], p["vp"], None)

    i[0].fill_(-1)
    assert write() == 0 and write(n=0, q=None) == 0
    for kw in (dict(n=-1), dict(qs=511), dict(qs=516), dict(ks=128), dict(vs=260), dict(q=None), dict(pos=None),
               dict(q=P(x) + 8), dict(kp=P(o[1]) + 2), dict(kp=P(o[2])), dict(qo=P(x)), dict(wq=P(x) + 4)):
        assert write(**kw) == -1, kw
    assert write(n=(1 << 24) + 1) == -4

    def attention(batch=1, n=1, **kw):
        p = dict(q=P(x), k=P(o[0]), v=P(o[1]), table=P(i[4]), start=P(i[5]), kv=P(i[6]), out=P(o[2]), lse=None)
        p.update(kw)
        return lib.wi_paged_attention(h, batch, n, p["q"], p["k"], p["v"], p["table"], p["start"], p["kv"], p["out"],
                                      p["lse"], None)

    assert attention() == 0 and attention(n=0, q=None) == 0
    for kw in (dict(batch=0), dict(batch=3), dict(n=-1), dict(q=None), dict(k=P(o[0]) + 8), dict(out=P(x)),
               dict(out=P(o[2]) + 4), dict(kv=P(i[6]) + 1), dict(lse=P(o[3]) + 2)):
        assert attention(**kw) == -1, kw
    assert attention(n=(1 << 24) + 1) == -4

    def gather(batch=1, layers=1, pos0=0, n=1, **kw):
        p = dict(k=P(o[0]), v=P(o[1]), ko=P(o[2]), vo=P(o[3]))
        p.update(kw)
        return lib.wi_paged_gather(h, batch, layers, p["k"], p["v"], P(i[4]), P(i[6]), pos0, n, p["ko"], p["vo"], None)

    assert gather() == 0 and gather(n=0, k=None) == 0
    for kw in (dict(batch=0), dict(batch=3), dict(layers=0), dict(pos0=-1), dict(n=-1), dict(n=65), dict(pos0=64),
               dict(k=None), dict(ko=P(o[3])), dict(ko=P(o[0])), dict(vo=P(o[3]) + 8)):
        assert gather(**kw) == -1, kw
    pc.check()

    t = torch.zeros
    dev = dict(dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="k_pages"):
        pc.attention(t((1, 4, 128), **dev), t((8, 2, 16, 64), **dev), o[1], i32([[0] * 4]), i32([0, 1]), i32([1]))
    with pytest.raises(ValueError, match="q "):
        pc.attention(t((1, 4, 128), device=DEV), o[0], o[1], i32([[0] * 4]), i32([0, 1]), i32([1]))
    with pytest.raises(ValueError, match="block_table"):
        pc.attention(t((2, 4, 128), **dev), o[0], o[1], i32([[0] * 4]), i32([0, 1, 2]), i32([1, 1]))
    with pytest.raises(ValueError, match="kv_len"):
        pc.attention(t((1, 4, 128), **dev), o[0], o[1], i32([[0] * 4]), i32([0, 1]), i32([1]).cpu())
    pc.free()


# ------------------------------------------------------------ all of them together ----

def model_step(pc, x, w, tb, pools, n):
    """One layer's step of a toy decoder: the given projections, cache write, attention."""
    hq, hkv = pc.n_q_heads, pc.n_kv_heads
    q, k, v = x.split([hq * 128, hkv * 128, hkv * 128], 1)
    q = pc.write(q.view(n, hq, 128), k.view(n, hkv, 128), v.view(n, hkv, 128), tb["positions"], tb["slots"], *pools,
                 q_weight=w[0], k_weight=w[1])
    return q, pc.attention(q, *pools, tb["block_table"], tb["q_start"], tb["kv_len"])


def test_serving_steps_then_index(wi):
    """Chunked prefill and single tokens of three requests through tables, write and attention, every step against
    the oracle over all the tokens so far; then an index built from the pages equals one built from the same rows
    laid out contiguously, and a step's token written without slots is appended to it."""
    rng = np.random.default_rng(20)
    hq, hkv, page, batch, f, eps = 8, 2, 16, 3, freqs(128), 1e-6
    n_pages, width = 250, 80
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, batch, width, inv_freq=f, eps=eps))
    pools = [torch.full((n_pages, hkv, page, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    w, W = zip(*(bf(1 + 0.2 * rng.normal(size=128)) for _ in range(2)))
    tb = {"block_table": i32(np.full((batch, width), -1))}
    free, n_free = i32(rng.permutation(n_pages)), i32([n_pages])
    kv = [0] * batch
    K, V = [np.zeros((0, hkv, 128)) for _ in range(batch)], [np.zeros((0, hkv, 128)) for _ in range(batch)]
    for new in [(100, 0, 33), (60, 700, 1), (1, 1, 1), (900, 350, 1024), (5, 3, 16)]:
        n = sum(new) + 2
        x, X = bf(rng.normal(size=(n, (hq + 2 * hkv) * 128)))
        for k, size in (("kv_len", batch), ("q_start", batch + 1), ("slots", n), ("positions", n)):
            tb[k] = i32([0] * size)
        left = i32([0])
        pc.tables(i32(kv), i32(new), free, n_free, tb["block_table"], tb["kv_len"], tb["q_start"], tb["slots"],
                  tb["positions"], left)
        q, out = model_step(pc, x, w, tb, pools, n)
        pc.check()
        n_free = left
        X = X.reshape(n, hq + 2 * hkv, 128)
        Q, at = f64(q), 0
        for b in range(batch):
            s = slice(at, at + new[b])
            pos = np.arange(kv[b], kv[b] + new[b])
            k, _ = paged.norm_rotate(X[s, hq:hq + hkv], W[1], eps, pos, f)
            K[b], V[b] = np.concatenate([K[b], k]), np.concatenate([V[b], X[s, hq + hkv:]])
            kv[b] += new[b]
            seen = np.arange(kv[b])[None] <= pos[:, None]
            for h in range(hq if new[b] else 0):
                sc = Q[s, h] @ K[b][:, h // 4].T / np.sqrt(128)
                p = np.where(seen, np.exp(sc - sc.max(1, keepdims=True, initial=-1e9)), 0)
                p /= p.sum(1, keepdims=True)
                # the cached keys are rounded to bf16: a score is off by up to 2^-8 |q||k| / sqrt(128) on top
                ds = 2.0 ** -8 * np.linalg.norm(Q[s, h], axis=-1) * np.linalg.norm(K[b][:, h // 4], axis=-1).max() / np.sqrt(128)
                err = np.abs(f64(out[s, h]) - p @ V[b][:, h // 4])
                assert (err <= (2.0 ** -7 + 2 * ds + 2.0 ** -10)[:, None] * (p @ np.abs(V[b][:, h // 4]))).all()
            at += new[b]
    # the index: the first 1024 positions of requests 0 and 1 through the pages, and laid out by hand
    two = [0, 1]
    rows = {}
    for name, pool in zip("kv", pools):
        P = pool.cpu()
        T = tb["block_table"].cpu()
        rows[name] = torch.stack([torch.cat([P[T[b, j]] for j in range(64)], 1) for b in two])[:, None].contiguous().to(DEV)
    cfg = wi.make_config(2, 1, hq, hkv, 1024, seg_len=512, clusters_per_seg=32, iters=2, max_append=4, budget_k=8)
    ix = wi.WaveIndex.build_paged(cfg, pc, pools[0], pools[1], tb["block_table"], tb["kv_len"][:2].contiguous())
    iy = wi.WaveIndex.build(cfg, rows["k"], rows["v"])
    one, _ = bf(rng.normal(size=(2, (hq + 2 * hkv) * 128)))
    q, k, v = one.split([hq * 128, hkv * 128, hkv * 128], 1)
    kn, vn = (torch.empty((2, hkv, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    qn = pc.write(q.view(2, hq, 128), k.view(2, hkv, 128), v.view(2, hkv, 128), i32([1024, 1024]), None, kn, vn,
                  q_weight=w[0], k_weight=w[1])
    for _ in range(2):
        a, b = ix.decode(qn, kn, vn), iy.decode(qn, kn, vn)
        assert torch.equal(a, b) and a.isfinite().all()
    ix.check()
    pc.check()
    # full attention over the index's cache stands beside full attention over the pages
    ks, vs = (torch.empty((2, 1, hkv, 1024, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pc.gather(pools[0], pools[1], tb["block_table"], tb["kv_len"][:2].contiguous(), 0, ks, vs)
    iz = wi.WaveIndex.build(cfg, ks, vs)
    dense = f64(iz.dense_decode(qn)).reshape(2, hq, 128)
    full = f64(pc.attention(qn, pools[0], pools[1], tb["block_table"], i32([0, 1, 2]), i32([1024, 1024])))
    # the page result is rounded to bf16 and so are its weights
    assert (np.abs(full - dense) <= 2.0 ** -8 * np.abs(dense) + 2.0 ** -7 * np.abs(f64(vs)).max()).all()
    for i in (ix, iy, iz):
        i.free()
    pc.free()


def test_captured_step_replays_over_new_contents(wi):
    """tables, write, attention and gather captured once on a stream of their own and replayed as the lengths and
    tokens change, against eager calls of another handle on the current stream."""
    rng = np.random.default_rng(21)
    hq, hkv, page, batch, n, n_pages, width = 28, 4, 16, 4, 40, 300, 70
    cfg = wi.make_paged_config(hq, hkv, page, n_pages, batch, width)
    free = i32(rng.permutation(n_pages))
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((n, (hq + 2 * hkv) * 128), dtype=torch.bfloat16, device=DEV)

    def fresh():
        s = {"pc": wi.PagedCache(cfg), "ctx": i32([0] * batch), "new": i32([0] * batch), "n_free": i32([n_pages]),
             "left": i32([0]), "out": torch.zeros((n, hq, 128), dtype=torch.bfloat16, device=DEV),
             "q": torch.zeros((n, hq, 128), dtype=torch.bfloat16, device=DEV),
             "tb": {"block_table": i32(np.full((batch, width), -1)), "kv_len": i32([0] * batch),
                    "q_start": i32([0] * (batch + 1)), "slots": i32([0] * n), "positions": i32([0] * n)},
             "pools": [torch.zeros((n_pages, hkv, page, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)],
             "rows": [torch.zeros((batch, 1, hkv, 33, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]}
        return s

    def step(s, stream=None):
        tb, pc = s["tb"], s["pc"]
        pc.tables(s["ctx"], s["new"], free, s["n_free"], tb["block_table"], tb["kv_len"], tb["q_start"], tb["slots"],
                  tb["positions"], s["left"], stream=stream)
        q, k, v = x.split([hq * 128, hkv * 128, hkv * 128], 1)
        pc.write(q.view(n, hq, 128), k.view(n, hkv, 128), v.view(n, hkv, 128), tb["positions"], tb["slots"], *s["pools"],
                 q_out=s["q"], q_weight=w, k_weight=w, stream=stream)
        pc.attention(s["q"], *s["pools"], tb["block_table"], tb["q_start"], tb["kv_len"], out=s["out"], stream=stream)
        pc.gather(*s["pools"], tb["block_table"], tb["kv_len"], 7, *s["rows"], stream=stream)

    a, b = fresh(), fresh()
    side = torch.cuda.Stream()
    step(a, side)                  # a step of no tokens: launches warmed up, nothing written
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(a)
    for new in [(30, 1, 0, 9), (1, 1, 1, 1), (0, 40, 0, 0), (10, 10, 10, 10), (1, 1, 1, 1)]:
        x.copy_(torch.from_numpy(rng.normal(size=x.shape).astype(np.float32)))
        for s in (a, b):
            s["new"].copy_(i32(new))
        torch.cuda.synchronize()
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        for s in (a, b):
            s["pc"].check()
            s["ctx"].copy_(s["tb"]["kv_len"])
            s["n_free"].copy_(s["left"])
        for k in a["tb"]:
            assert torch.equal(a["tb"][k], b["tb"][k]), k
        for k in ("pools", "rows"):
            assert all(torch.equal(u, v) for u, v in zip(a[k], b[k])), k
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["q"], b["q"])
    del graph
    for s in (a, b):
        s["pc"].free()


# ------------------------------------------------------------ calls that overlap, repeat and share ----

def test_attention_long_chunks(wi):
    """More blocks than one CTA takes, several items to a CTA, items cut in two and in many."""
    attention_case(wi, 8, 2, 64, [700, 1, 513], [5700, 9000, 3513], seed=30)
    attention_case(wi, 4, 1, 16, [64], [20064], seed=31)
    attention_case(wi, 28, 4, 128, [37, 300], [4037, 6300], seed=32)


@pytest.mark.parametrize("order", ["rising", "falling", "late"])
def test_attention_maxima_that_move_far(wi, order):
    """Scores that outgrow everything before them block after block (by thousands), fall, or come late: the weights'
    reference has to follow."""
    hq, hkv, n, kv, page = 4, 1, 40, 900, 16
    rng = np.random.default_rng(33)
    table, n_pages = lay_out([kv], page, rng)
    base = rng.normal(size=128)
    q, Q = bf(np.broadcast_to(base * 4, (n, hq, 128)) + rng.normal(size=(n, hq, 128)))
    size = {"rising": np.linspace(-3, 3, kv) ** 3, "falling": -np.linspace(-3, 3, kv) ** 3,
            "late": np.where(np.arange(kv) < 700, -20.0, 1.0)}[order]
    K = base * size[:, None] + 0.1 * rng.normal(size=(kv, 128))
    Kp, Vp = np.zeros((n_pages, hkv, page, 128)), rng.normal(size=(n_pages, hkv, page, 128))
    for p in range(kv):
        Kp[table[0, p // page], 0, p % page] = K[p]
    k, Kr = bf(Kp)
    v, Vr = bf(Vp)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 1, table.shape[1]))
    lse = torch.empty((n, hq), device=DEV)
    out = pc.attention(q, k, v, i32(table), i32([0, n]), i32([kv]), lse=lse)
    pc.check()
    ref, rlse, spread = paged.attention(Q, Kr, Vr, table, [0, n], [kv])
    top = np.linalg.norm(Q, axis=-1) * np.sqrt((Kr ** 2).sum(-1).max()) / np.sqrt(128)
    ds = 128 * 2.0 ** -24 * top + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -7) * spread * (2.0 ** -8 + 2 * ds + kv * 2.0 ** -23)[..., None]
    assert (np.abs(f64(out) - ref) <= tol).all()
    assert (np.abs(f64(lse) - rlse) <= ds + kv * 2.0 ** -24 + 2.0 ** -22 * np.abs(rlse) + 2.0 ** -20).all()
    pc.free()


def test_attention_requests_that_share_pages(wi):
    """Two requests with a common prefix held once."""
    rng = np.random.default_rng(34)
    k, K = bf(rng.normal(size=(12, 2, 16, 128)))
    v, V = bf(rng.normal(size=(12, 2, 16, 128)))
    table = [[3, 1, 4, 5, 9], [3, 1, 4, 2, 6], [3, 1, 4, 5, 9]]
    q, Q = bf(rng.normal(size=(22, 8, 128)))
    pc = wi.PagedCache(wi.make_paged_config(8, 2, 16, 12, 3, 5))
    out = pc.attention(q, k, v, i32(table), i32([0, 20, 21, 22]), i32([70, 66, 51]))
    pc.check()
    ref, _, spread = paged.attention(Q, K, V, table, [0, 20, 21, 22], [70, 66, 51])
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread).all()
    pc.free()


def test_attention_calls_in_turn_and_on_two_streams(wi):
    """One handle used for single tokens and chunks in turn, many times, and two handles at once on two streams:
    always the same bits."""
    rng = np.random.default_rng(35)
    kv = [3000, 2000, 700]
    table, n_pages = lay_out(kv, 16, rng)
    k, v = (bf(rng.normal(size=(n_pages, 2, 16, 128)))[0] for _ in range(2))
    pcs = [wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, 3, table.shape[1])) for _ in range(2)]
    jobs = []
    for new in [(1, 0, 0), (1, 1, 1), (0, 200, 90), (2, 0, 0), (150, 1, 33)]:
        q = bf(rng.normal(size=(sum(new), 8, 128)))[0]
        jobs.append((q, k, v, i32(table), i32(np.concatenate([[0], np.cumsum(new)])), i32(kv)))
    first = [pcs[0].attention(*j) for j in jobs]
    torch.cuda.synchronize()
    for _ in range(20):
        for j, f in zip(jobs, first):
            assert torch.equal(pcs[0].attention(*j), f)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(f) for _ in range(10) for f in first] for _ in range(2)]
    for i in range(len(outs[0])):
        for s in range(2):
            n = i if s == 0 else len(outs[0]) - 1 - i   # different jobs at the same time
            pcs[s].attention(*jobs[n % len(jobs)], out=outs[s][n], stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        for n, o in enumerate(outs[s]):
            assert torch.equal(o, first[n % len(jobs)])
        pcs[s].check()
        pcs[s].free()


def test_calls_refuse_shared_memory(wi):
    pc = wi.PagedCache(wi.make_paged_config(4, 2, 16, 8, 2, 4))
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((4, 8 * 128), **bf16)
    q, k, v = (t.view(4, -1, 128) for t in x.split([512, 256, 256], 1))
    pools = [torch.zeros((8, 2, 16, 128), **bf16) for _ in range(2)]
    neg, flat = i32([-1] * 4), torch.zeros(4 * 1024, **bf16)
    for kw in (dict(q_out=x.view(-1)[:2048].view(4, 4, 128)),            # the fused rows, other strides
               dict(q_out=pools[0].view(-1)[:2048].view(4, 4, 128))):
        with pytest.raises(wi.WiError, match="shares memory"):
            pc.write(q, k, v, neg, neg, *pools, **kw)
    kn = flat[:1024].view(4, 2, 128)
    with pytest.raises(wi.WiError, match="shares memory"):               # keys and values half a buffer apart
        pc.write(q, k, v, neg, None, kn, flat[512:1536].view(4, 2, 128))
    table, start, kv = i32([[0] * 4]), i32([0, 4]), i32([4])
    qc = torch.zeros((4, 4, 128), **bf16)
    with pytest.raises(wi.WiError, match="shares memory"):
        pc.attention(qc, *pools, table, start, kv, out=pools[1].view(-1)[:2048].view(4, 4, 128))
    with pytest.raises(wi.WiError, match="shares memory"):
        pc.attention(qc, *pools, table, start, kv, lse=qc.view(torch.float32).view(-1)[:16].view(4, 4))
    big = torch.zeros((1, 1, 2, 8, 128), **bf16)
    with pytest.raises(wi.WiError, match="shares memory"):
        pc.gather(*pools, table, kv, 0, big, pools[0].view(-1)[2048:4096].view(1, 1, 2, 8, 128))
    i = i32(range(40))
    with pytest.raises(wi.WiError, match="shares memory"):
        pc.tables(i[0:1], i[1:2], i[2:4], i[4:5], i[5:9].view(1, 4), i[9:10], i[10:12], i[12:14], i[13:15], i[20:21])
    pc.check()
    pc.free()


def test_write_then_attention_of_one_token_many_times(wi):
    """A decode loop without any wait in between: each step's token is written and attended to before the next one,
    kernel chained to kernel; against the same loop with a wait after every call."""
    rng = np.random.default_rng(36)
    hq, hkv, page, steps = 8, 2, 16, 60
    cfg = wi.make_paged_config(hq, hkv, page, 40, 2, 20)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    x = torch.from_numpy(rng.normal(size=(steps, 2, (hq + 2 * hkv) * 128)).astype(np.float32)).to(DEV).bfloat16()

    def loop(wait):
        pc = wi.PagedCache(cfg)
        pools = [torch.zeros((40, hkv, page, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        table, free = i32(np.full((2, 20), -1)), i32(np.random.default_rng(1).permutation(40))
        ctx, left = [i32([200, 7]), i32([0, 0])], [i32([40]), i32([0])]
        start, slots, pos, one = i32([0, 0, 0]), i32([0, 0]), i32([0, 0]), i32([1, 1])
        # the positions before the first step: their pages, and zeros in them
        pc.tables(i32([0, 0]), ctx[0], free, left[0], table, ctx[1], i32([0, 0, 0]), i32([0] * 207), i32([0] * 207), left[1])
        left.reverse()
        outs = []
        for t in range(steps):
            pc.tables(ctx[0], one, free, left[0], table, ctx[1], start, slots, pos, left[1])
            q, k, v = x[t].split([hq * 128, hkv * 128, hkv * 128], 1)
            q = pc.write(q.view(2, hq, 128), k.view(2, hkv, 128), v.view(2, hkv, 128), pos, slots, *pools, None, w, w)
            outs.append(pc.attention(q, *pools, table, start, ctx[1]))
            ctx.reverse()
            left.reverse()
            if wait:
                torch.cuda.synchronize()
        pc.check()
        pc.free()
        return torch.stack(outs), pools

    a, b = loop(False), loop(True)
    assert torch.equal(a[0], b[0]) and all(torch.equal(u, v) for u, v in zip(a[1], b[1]))


def test_a_freed_cache_refuses_its_calls(wi):
    pc = wi.PagedCache(wi.make_paged_config(4, 2, 16, 8, 2, 4))
    x = torch.zeros((8, 2, 16, 128), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device=DEV)
    args = (q, x, x.clone(), i32([[0] * 4]), i32([0, 1]), i32([1]))
    pc.attention(*args)
    pc.check()
    pc.free()
    with pytest.raises(ValueError, match="freed"):
        pc.attention(*args)
    pc.free()   # once more is no error


@pytest.mark.parametrize("value", [np.nan, np.inf, 3e38])
def test_attention_rows_do_not_touch_each_other(wi, value):
    """A token whose query is broken, or whose scores outgrow everything, leaves every other row's bits as they are."""
    rng = np.random.default_rng(37)
    kv = [700, 300]
    table, n_pages = lay_out(kv, 16, rng)
    k, v = (bf(rng.normal(size=(n_pages, 2, 16, 128)))[0] for _ in range(2))
    q = bf(rng.normal(size=(151, 8, 128)))[0]
    args = (k, v, i32(table), i32([0, 150, 151]), i32(kv))
    pc = wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, 2, table.shape[1]))
    a = pc.attention(q, *args)
    q2 = q.clone()
    q2[77, 3] = value
    b = pc.attention(q2, *args)
    pc.check()
    same = torch.ones((151, 8), dtype=torch.bool, device=DEV)
    same[77, 3] = False
    assert torch.equal(a[same], b[same]) and not torch.equal(a[77, 3], b[77, 3])
    pc.free()


def test_captured_behind_copies_and_joins(wi):
    """In a graph: behind a memory copy, behind a fork and a join of two streams, and the same eagerly behind events:
    each kernel may be scheduled early, and still waits for what it reads."""
    rng = np.random.default_rng(38)
    hq, hkv, page, n = 8, 2, 16, 300
    table, n_pages = lay_out([2300, 40], page, rng)
    cfg = wi.make_paged_config(hq, hkv, page, n_pages, 2, table.shape[1])
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    src = bf(rng.normal(size=(n, (hq + 2 * hkv) * 128)))[0]
    old = [bf(rng.normal(size=(n_pages, hkv, page, 128)))[0] for _ in range(2)]
    slots = np.concatenate([[table[0, p // page] * page + p % page for p in range(2000, 2299)], [table[1, 2] * page + 7]])
    pos = np.concatenate([np.arange(2000, 2299), [39]])
    args = (i32(table), i32([0, 299, 300]), i32([2299, 40]))
    pos, slots = i32(pos), i32(slots)

    def make():
        s = {"pc": wi.PagedCache(cfg), "x": torch.zeros_like(src), "pools": [torch.zeros_like(o) for o in old],
             "q": torch.zeros((n, hq, 128), **bf16), "out": torch.zeros((n, hq, 128), **bf16),
             "rows": [torch.zeros((2, 1, hkv, 40, 128), **bf16) for _ in range(2)]}
        return s

    def step(s, main, side):
        for a, b in zip(s["pools"], old):
            a.copy_(b)
        s["x"].copy_(src)                                   # a copy, not a kernel
        q, k, v = s["x"].split([hq * 128, hkv * 128, hkv * 128], 1)
        s["pc"].write(q.view(n, hq, 128), k.view(n, hkv, 128), v.view(n, hkv, 128), pos, slots, *s["pools"], s["q"])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            s["pc"].gather(*s["pools"], args[0], args[2], 0, *s["rows"])
        s["pc"].attention(s["q"], *s["pools"], *args, out=s["out"])
        main.wait_stream(side)
        # behind the join: over what both branches left
        s["pc"].gather(*s["pools"], args[0], args[2], 0, *s["rows"])

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    eager, captured = make(), make()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        step(eager, main, side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        step(captured, main, side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    plain = make()                                          # one call at a time
    for a, b in zip(plain["pools"], old):
        a.copy_(b)
    q, k, v = src.split([hq * 128, hkv * 128, hkv * 128], 1)
    for call in (lambda: plain["pc"].write(q.view(n, hq, 128), k.view(n, hkv, 128), v.view(n, hkv, 128), pos, slots,
                                           *plain["pools"], plain["q"]),
                 lambda: plain["pc"].attention(plain["q"], *plain["pools"], *args, out=plain["out"]),
                 lambda: plain["pc"].gather(*plain["pools"], args[0], args[2], 0, *plain["rows"])):
        torch.cuda.synchronize()
        call()
    torch.cuda.synchronize()
    for s in (eager, captured):
        s["pc"].check()
        assert torch.equal(s["q"], plain["q"]) and torch.equal(s["out"], plain["out"])
        for k in ("pools", "rows"):
            assert all(torch.equal(a, b) for a, b in zip(s[k], plain[k]))
    del graph
    for s in (eager, captured, plain):
        s["pc"].free()


def test_written_tokens_feed_the_decode_step(wi):
    """Steps of an index whose query and new row a cache's write makes just before, back to back and (without the
    appended row: an appending step is not for a graph) captured, equal the same steps taken one call at a time."""
    rng = np.random.default_rng(39)
    hq, hkv, batch, ctx, steps = 8, 2, 2, 1024, 12
    cfg = wi.make_config(batch, 1, hq, hkv, ctx, seg_len=512, clusters_per_seg=32, iters=2, max_append=2 * steps,
                         budget_k=8)
    ks, vs = (bf(rng.normal(size=(batch, 1, hkv, ctx, 128)))[0] for _ in range(2))
    xs = [bf(rng.normal(size=(batch, (hq + 2 * hkv) * 128)))[0] for _ in range(steps)]
    f = freqs(128)
    results = []
    for wait, append in ((True, True), (False, True), (True, False), ("graph", False)):
        pc = wi.PagedCache(wi.make_paged_config(hq, hkv, 16, 4, batch, 4, inv_freq=f))
        ix = wi.WaveIndex.build(cfg, ks.clone(), vs.clone())  # a build reorders the rows in place
        qn = torch.zeros((batch, hq, 128), dtype=torch.bfloat16, device=DEV)
        kn, vn = (torch.zeros((batch, hkv, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        pos, at = [i32([ctx + i] * batch) for i in range(steps)], i32([0] * batch)
        buf = torch.zeros_like(xs[0])

        def step(x, at):
            q, k, v = x.split([hq * 128, hkv * 128, hkv * 128], 1)
            pc.write(q.view(batch, hq, 128), k.view(batch, hkv, 128), v.view(batch, hkv, 128), at, None, kn, vn, qn)
            if wait is True:
                torch.cuda.synchronize()
            return ix.decode(qn, kn, vn) if append else ix.decode(qn)

        outs = []
        if wait == "graph":
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = step(buf, at)
            for x, p in zip(xs, pos):
                buf.copy_(x)
                at.copy_(p)
                graph.replay()
                outs.append(out.clone())
            torch.cuda.synchronize()
            del graph
        else:
            outs = [step(x, p).clone() for x, p in zip(xs, pos)]
        torch.cuda.synchronize()
        ix.check()
        pc.check()
        results.append(torch.stack(outs))
        ix.free()
        pc.free()
    assert results[0].isfinite().all() and results[2].isfinite().all() and not torch.equal(results[0], results[2])
    assert torch.equal(results[0], results[1]) and torch.equal(results[2], results[3])


def test_largest_batch(wi):
    """4096 requests in one call of each operator that takes a batch, every fifth of them without a token."""
    rng = np.random.default_rng(40)
    batch, hq, hkv, page, width = 4096, 2, 1, 16, 3
    n_pages = batch * width
    kv = rng.integers(0, page * (width - 1), size=batch)
    new = np.where(np.arange(batch) % 5 == 4, 0, rng.integers(1, 4, size=batch))
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, batch, width))
    order = rng.permutation(n_pages)
    have = -(-kv // page)
    table = np.full((batch, width), -1)
    at = 0
    for b in range(batch):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    n = int(new.sum())
    t = {k: i32([0] * s) for k, s in (("kv", batch), ("qs", batch + 1), ("slots", n), ("pos", n), ("left", 1))}
    T = i32(table)
    pc.tables(i32(kv), i32(new), i32(order[at:]), i32([n_pages - at]), T, t["kv"], t["qs"], t["slots"], t["pos"], t["left"])
    pc.check()
    pools, F = zip(*(bf(rng.normal(size=(n_pages, hkv, page, 128))) for _ in range(2)))
    q, Q = bf(rng.normal(size=(n, hq, 128)))
    out = f64(pc.attention(q, *pools, T, t["qs"], t["kv"]))
    pc.check()
    TT, qs = T.cpu().numpy(), np.concatenate([[0], np.cumsum(new)])
    assert (t["qs"].cpu().numpy() == qs).all() and (t["kv"].cpu().numpy() == kv + new).all()
    for b in range(batch):
        total = kv[b] + new[b]
        K, V = (x.reshape(n_pages, page, 128)[TT[b, :-(-total // page)]].reshape(-1, 128)[:total] for x in F)
        for i in range(new[b]):
            see = kv[b] + i + 1
            s = Q[qs[b] + i] @ K[:see].T / np.sqrt(128)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            # weights and result are rounded to bf16, each by at most half a step (2^-8); a score of at most 30 in 32
            # bits is off by 128 2^-24 30 = 2^-12.1 at most, its weight by twice that
            bound = (2.0 ** -7 + 2.0 ** -11) * (p @ np.abs(V[:see])) + 1e-6
            assert (np.abs(out[qs[b] + i] - p @ V[:see]) <= bound).all(), b
    pc.free()


@pytest.mark.parametrize("hq,hkv,new,kv", [
    (32, 8, [5], [305]), (32, 8, [1], [512]), (32, 8, [1], [513]), (32, 8, [8], [512]), (32, 8, [8], [514]),   # one request whole and cut
    (64, 64, [1], [300]), (200, 200, [2], [400]), (8, 1, [4], [6000]), (28, 4, [4], [5000]), (4, 1, [8], [20000]),
    (32, 8, [2, 3, 0, 1], [900, 4000, 0, 9]), (6, 2, [1] * 10, [700] * 10), (32, 8, [8], [1]),       # 32 rows and fewer
    (32, 8, [9], [300]), (4, 1, [9], [20000]), (28, 4, [5, 30, 1], [4000, 9000, 3000]), (8, 8, [33], [7000]),  # and more
    (4, 2, [130, 17, 2], [5000, 2500, 9000])])
def test_attention_parts_of_few_and_many_rows(wi, hq, hkv, new, kv):
    """Items cut into a few or dozens of parts, of one to 128 rows, merged in the kernel or by one of its own."""
    attention_case(wi, hq, hkv, 16, new, [max(a, b) for a, b in zip(kv, new)], seed=sum(kv) + sum(new))


@pytest.mark.parametrize("hq,hkv,new,kv", [
    (32, 8, [1] * 32, [700] * 32), (32, 8, [1] * 33, [700] * 33), (28, 4, [1] * 18, [2500] * 18), (12, 2, [1] * 21, [1500] * 21),
    (4, 1, [20] + [0] * 19, [6000] + [0] * 19), (4, 1, [0] * 5 + [30, 2] + [0] * 25, [50] * 5 + [9000, 4000] + [0] * 25),
    (8, 2, [3, 0, 5, 0, 1, 0, 2, 1, 0, 0, 4, 0], [2000] * 12), (1, 1, [1] * 128, [500] * 128), (1, 1, [128] + [0] * 127, [3000] + [0] * 127)])
def test_attention_no_more_tokens_than_requests(wi, hq, hkv, new, kv):
    """Steps of single tokens, and calls that look like one by their sizes while some requests have several tokens."""
    attention_case(wi, hq, hkv, 16, new, kv, seed=sum(kv) + len(new))
