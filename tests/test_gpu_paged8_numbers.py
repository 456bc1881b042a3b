"""Numbers at the ends of what the paged cache in 8 bits holds: queries of nothing, scales far apart, weights far below the
row's largest, sums over long contexts.  Tolerances as tests/test_gpu_paged8.py derives them, unless said."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import DEV, bf, f64, i32, lay_out
from test_gpu_paged8 import as_scales, as_values, compare, exps8, random_pool, upload, values8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wi():
    import clustered_sparse_kv_gb300 as m
    return m


def attend(wi, Q, pools, table, start, kv, page):
    """out and lse of attention8 in 64 bits; queries in bf16, pools as (values, exponents)."""
    n, hq = Q.shape[:2]
    (k, ks), (v, vs) = pools
    pc = wi.PagedCache(wi.make_paged_config(hq, k.shape[1], page, k.shape[0], len(kv), table.shape[1]))
    out = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n, hq), 7.0, device=DEV)
    pc.attention8(Q, k, v, ks, vs, i32(table), i32(start), i32(kv), out=out, lse=lse)
    pc.check()
    pc.free()
    return f64(out), f64(lse)


# ------------------------------------------------------------ queries of nothing ----

@pytest.mark.parametrize("new,ctx", [([1], [40]), ([40], [0]), ([40], [75]), ([7, 1, 100], [0, 30, 300]), ([300], [0])])
def test_attention8_of_zeros_that_were_written(wi, new, ctx):
    """A call on zeroed rows, as a warm-up's or a padded batch's: groups of zero keys have the smallest scale, and every row is
    the mean of the values that it sees."""
    rng = np.random.default_rng(70)
    hq, hkv, page = 8, 2, 16
    kv = [c + n for c, n in zip(ctx, new)]
    table, n_pages = lay_out(kv, page, rng)
    start = np.concatenate([[0], np.cumsum(new)])
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, len(kv), table.shape[1]))
    pools = [torch.zeros((n_pages, hkv, page, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
    pools += [torch.zeros((n_pages, hkv, 1), dtype=torch.uint8, device=DEV) for _ in range(2)]
    at = np.concatenate([np.arange(n) for n in kv])          # everything that is cached, in one write
    who = np.repeat(np.arange(len(kv)), kv)
    slots = table[who, at // page] * page + at % page
    zeros = torch.zeros((len(at), hq, 128), dtype=torch.bfloat16, device=DEV)
    v, V = bf(rng.normal(size=(len(at), hkv, 128)))
    q = pc.write8(zeros, zeros[:, :hkv], v, i32(at), i32(slots), *pools)
    assert (exps8(pools[2])[table[table >= 0]] == paged.LOWEST).all()
    q = q[:start[-1]].contiguous()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    pc.attention8(q, *pools, i32(table), i32(start), i32(kv), out=out, lse=lse)
    pc.check()
    pc.free()
    K, V = (paged.widened(values8(p), exps8(s)) for p, s in (pools[::2], pools[1::2]))
    compare(f64(out), f64(lse), f64(q), K, V, table, start, kv)


@pytest.mark.parametrize("size", [0.0, 2.0 ** -126, 2.0 ** -100, 2.0 ** -60, 2.0 ** -15, 1.0])
@pytest.mark.parametrize("exps", [[-64], [-127], [-127, 0], [-64, -22, 3]])
@pytest.mark.parametrize("new,kv", [([50], [50]), ([50, 3, 200], [300, 3, 333]), ([1, 1], [100, 130])])
def test_attention8_of_small_queries_over_small_scales(wi, size, exps, new, kv):
    """Factors of a score that vanish: the row's and the group's together leave fp32, in groups that a row sees and in those
    that it does not.  Rows of zeros beside others."""
    rng = np.random.default_rng(71)
    hq, hkv, page = 8, 2, 32
    table, n_pages = lay_out(kv, page, rng)
    start = np.concatenate([[0], np.cumsum(new)])
    Q = rng.normal(size=(start[-1], hq, 128)) * size
    Q[::3, ::2] = 0
    q, Q = bf(Q)
    values = [paged.e4m3(rng.normal(size=(n_pages, hkv, page, 128)) * 50) for _ in range(2)]
    e = rng.choice(exps, (n_pages, hkv, page // 16))
    pools = [(values[0], e), (values[1], np.full_like(e, -6))]
    out, lse = attend(wi, q, [upload(p) for p in pools], table, start, kv, page)
    compare(out, lse, Q, *(paged.widened(*p) for p in pools), table, start, kv)


# ------------------------------------------------------------ weights far below the largest ----

def behind_a_sink(wi, hq, tokens, requests, where, least):
    """One position of value 0, which weighs e^gap as much as any other, all alike and of value 1: what is left of a row is a
    multiple of one weight, whose rounding shows as it is.  Gaps from 0.3 to 18 (2^26) in steps that fall between rounding
    points, one for every row.  As many requests as leave their runs whole: a part that does not hold the sink would hold its
    weights better."""
    rng = np.random.default_rng(72)
    kv, page = 20000 + tokens, 16
    table, n_pages = lay_out([kv], page, rng)
    n = tokens * requests
    gaps = np.linspace(0.3, 18.0, n * hq).reshape(n, hq)
    base = np.sqrt(18.0 * np.sqrt(128) / 128)                   # of the sink's key: q . k = gap * sqrt(128)
    k0 = paged.e4m3(np.full(128, base * 64)) / 64
    q, Q = bf(np.broadcast_to((gaps * np.sqrt(128) / k0.sum())[..., None], (n, hq, 128)))
    pools = [(np.zeros((n_pages, 1, page, 128)), np.full((n_pages, 1, 1), -6)) for _ in range(2)]
    pools[1][0][table[0]] = 64
    pools[0][0][table[0, where // page], 0, where % page] = k0 * 64
    pools[1][0][table[0, where // page], 0, where % page] = 0
    start, lengths = np.arange(requests + 1) * tokens, [kv] * requests
    out, lse = attend(wi, q, [upload(p) for p in pools], np.repeat(table, requests, 0), start, lengths, page)
    gap = Q[..., 0] * k0.sum() / np.sqrt(128)
    others = kv - tokens + np.tile(np.arange(tokens), requests)[:, None]      # positions beside the sink
    ref = others / (others + np.exp(gap))
    # A weight is known to 2^-11 of itself or to `least` of the row's largest.  A score, of products that are all alike and exact in
    # pieces, is off by 128 * 2^-24 of itself, and its weight by as much; the tensor cores' 160 blocks of eight additions by 2^-23
    # each; a power of two and the sums of the weights by 2^-17; the output is rounded to bf16, 2^-8.
    tol = 2.0 ** -8 + 2.0 ** -11 + least * np.exp(gap) + 2 * 128 * 2.0 ** -24 * gap + 160 * 8 * 2.0 ** -23 + 2.0 ** -17
    err = np.abs(out / ref[..., None] - 1)
    assert (err <= tol[..., None]).all(), (err / tol[..., None]).max()
    assert (np.abs(lse - np.log(others + np.exp(gap))) <= 2.0 ** -11).all()


@pytest.mark.parametrize("where", [0, 3000, 19990])
@pytest.mark.parametrize("hq", [4, 8])
def test_attention8_weights_behind_a_sink_single_tokens(wi, hq, where):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    behind_a_sink(wi, hq, 1, 2 * sms, where, 2.0 ** -33)


@pytest.mark.parametrize("where", [0, 3000, 19990])
@pytest.mark.parametrize("hq,tokens", [(4, 44), (8, 3), (1, 200)])
def test_attention8_weights_behind_a_sink_chunks(wi, hq, tokens, where):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    behind_a_sink(wi, hq, tokens, sms, where, 2.0 ** -29)


# ------------------------------------------------------------ sums over long contexts ----

def test_attention8_single_tokens_sums_of_one_sign(wi):
    """What the tensor cores' additions cut off, over 2^18 positions in one CTA's run, on the average over many rows: less than
    an addition's 2^-23 of the sum for each of the 256 blocks of four that are added up there."""
    rng = np.random.default_rng(73)
    kv, batch = 1 << 18, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    pages = rng.integers(0, 8, kv // 128)
    q, Q = bf(rng.normal(size=(batch, 1, 128)))
    pools = [(paged.e4m3(rng.normal(size=(8, 1, 128, 128)) * 64), np.full((8, 1, 8), -6)),
             (paged.e4m3(rng.uniform(48, 80, size=(8, 1, 128, 128))), np.full((8, 1, 8), -6))]
    out, _ = attend(wi, q, [upload(p) for p in pools], np.repeat(pages[None], batch, 0), np.arange(batch + 1), [kv] * batch, 128)
    K, V = (paged.widened(*p).reshape(-1, 128) for p in pools)
    x = Q[:, 0] @ K.T / np.sqrt(128)
    w = np.repeat(np.bincount(pages, minlength=8), 128) * np.exp(x - x.max(1, keepdims=True))
    ref = w / w.sum(1, keepdims=True) @ V
    # 39000 elements, of which a few in a hundred round the other way by 2^-8: their mean is known to 2^-16
    bias = ((out[:, 0] - f64(torch.from_numpy(ref).bfloat16())) / ref).mean()
    assert abs(bias) <= 256 * 4 * 2.0 ** -23 + 2.0 ** -16, bias
