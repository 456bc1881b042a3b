"""Corners of the paged cache on the GPU: scores of minus infinity, rows that no token owns, bad offsets, handles and
streams.  Tolerances as tests/test_gpu_paged.py derives them."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import DEV, bf, f64, i32, lay_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wi():
    import clustered_sparse_kv_gb300 as m
    return m


# ------------------------------------------------------------ scores of minus infinity ----

@pytest.mark.parametrize("hq,hkv,batch,new,kv,hidden", [
    (4, 1, 1, 1, 380, 128),        # one tile, whole: the first block of one of its two chains
    (4, 1, 1, 1, 380, 256),        # ... of both
    (4, 1, 1, 40, 900, 128),       # two tiles, a block to a CTA
    (4, 1, 200, 40, 900, 128),     # two tiles, whole and cut at any block
    (4, 1, 200, 40, 900, 300),
    (8, 2, 1, 1, 20000, 12000),    # one tile, cut into many parts, some of which see nothing else
    (8, 2, 40, 1, 20000, 12000),   # ... into parts of several blocks
    (4, 1, 30, 300, 3000, 1500),   # several pairs of tiles
    (7, 1, 150, 20, 700, 300),     # rows that no token owns in every tile
    (4, 1, 100, 300, 300, 128),    # rows that see hidden positions only: as if they saw nothing
])
def test_attention_behind_scores_of_minus_infinity(wi, hq, hkv, batch, new, kv, hidden):
    """Keys with an element of minus infinity at positions 0 .. hidden - 1, which every query weights with nothing, and
    logits around -100 behind them: far below what 32 bits hold as a weight on their own.  The requests of a call are
    alike and share their pages."""
    rng = np.random.default_rng(kv + hidden)
    page = 16
    table, n_pages = lay_out([kv], page, rng)
    base = rng.normal(size=128)
    base[5] = 0.0
    base *= np.sqrt(128) / np.linalg.norm(base)
    q = np.broadcast_to(base * 3, (new, hq, 128)) + 0.3 * rng.normal(size=(new, hq, 128))
    q[..., 5] = 1.0
    rows = -base * 2.95 + 0.3 * rng.normal(size=(hkv, kv, 128))     # 3 * -2.95 * 128 / sqrt(128) = -100
    rows[:, :hidden, 5] = -np.inf
    rows[:, hidden:, 5] = 0.0
    Kp, Vp = np.zeros((n_pages, hkv, page, 128)), rng.normal(size=(n_pages, hkv, page, 128))
    for p in range(kv):
        Kp[table[0, p // page], :, p % page] = rows[:, p]
    (q, Q), (k, K), (v, V) = bf(q), bf(Kp), bf(Vp)
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, batch, table.shape[1]))
    lse = torch.empty((batch * new, hq), device=DEV)
    out = pc.attention(q.repeat(batch, 1, 1), k, v, i32(table.repeat(batch, 0)), i32(np.arange(batch + 1) * new),
                       i32([kv] * batch), lse=lse)
    pc.check()
    pc.free()
    out, lse = f64(out).reshape(batch, new, hq, 128), f64(lse).reshape(batch, new, hq)
    ref, rlse, spread = paged.attention(Q, K, V, table, [0, new], [kv])
    finite = np.where(np.isfinite(K), K, 0)
    top = np.linalg.norm(Q, axis=-1) * np.sqrt((finite ** 2).sum(-1).max()) / np.sqrt(128)
    ds = 128 * 2.0 ** -24 * top + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -7) * spread * (2.0 ** -8 + 2 * ds + kv * 2.0 ** -23)[..., None]
    assert (np.abs(out - ref) <= tol).all()
    none = np.arange(new) + kv - new < hidden
    assert (ref[none] == 0).all() and (rlse[none] == -np.inf).all() and (lse[:, none] == -np.inf).all()
    assert (rlse[~none] < -80).all()
    ltol = ds + kv * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(rlse), rlse, 0)) + 2.0 ** -20
    assert (np.abs(lse[:, ~none] - rlse[~none]) <= ltol[~none]).all()


# ------------------------------------------------------------ rows that no token owns ----

def test_attention_does_not_wait_for_rows_that_no_token_owns(wi):
    """NaN in the queries behind the last token: the same bits in the tokens' rows, and no block of theirs done twice
    (2040 tokens behind 14K positions took 1.4 times as long, 446 us to 320)."""
    rng = np.random.default_rng(50)
    hq, hkv, page, new, kv, n = 32, 8, 128, 2040, 16384, 2048
    table, n_pages = lay_out([kv], page, rng)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(50)
    k, v, q = (torch.randn(s, generator=gen, device=DEV, dtype=torch.bfloat16)
               for s in ((n_pages, hkv, page, 128), (n_pages, hkv, page, 128), (n, hq, 128)))
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, 1, table.shape[1]))
    args = (k, v, i32(table), i32([0, new]), i32([kv]))
    outs = [torch.zeros_like(q) for _ in range(2)]
    qs = [q.clone(), q.clone()]
    qs[0][new:] = 0
    qs[1][new:] = float("nan")
    times = [[], []]
    for turn in range(12):
        for s in range(2):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            for _ in range(5):
                pc.attention(qs[s], *args, out=outs[s])
            e[1].record()
            torch.cuda.synchronize()
            times[s].append(e[0].elapsed_time(e[1]))
    pc.check()
    pc.free()
    assert torch.equal(outs[0], outs[1]) and (outs[0][new:] == 0).all()
    zero, nan = (float(np.median(t[2:])) for t in times)
    assert nan < 1.2 * zero, (zero, nan)


# ------------------------------------------------------------ handles and streams ----

def test_a_new_cache_is_ready_for_every_stream(wi):
    """A cache made while the default stream is busy, over memory that was not zero, and used at once on a stream that
    does not wait for the default one: its tickets and error word are clear when the call that makes it returns."""
    rng = np.random.default_rng(51)
    kv, side = 20000, torch.cuda.Stream()
    table, n_pages = lay_out([kv], 16, rng)
    q, k, v = (bf(rng.normal(size=s))[0] for s in ((1, 8, 128), (n_pages, 2, 16, 128), (n_pages, 2, 16, 128)))
    args = (q, k, v, i32(table), i32([0, 1]), i32([kv]))
    outs = [torch.zeros_like(q) for _ in range(2)]
    dirt = torch.full((1 << 26,), -1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    del dirt
    torch.cuda.empty_cache()
    torch.cuda._sleep(400_000_000)          # about 0.2 s of work on the default stream
    pc = wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, 1, table.shape[1]))
    assert torch.cuda.default_stream().query()   # what clears them stands behind that work, and has been waited for
    pc.attention(*args, out=outs[0], stream=side)
    side.synchronize()
    pc.check()
    pc.attention(*args, out=outs[1])
    pc.check()
    pc.free()
    assert torch.equal(*outs) and (outs[0] != 0).any()


def test_a_reported_error_is_cleared_before_the_next_call(wi):
    """The check that reports an error clears it before it returns: one that a call on another stream meets right
    behind it is kept."""
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 4, 1, 4))
    side = torch.cuda.Stream()
    k, out = (torch.ones((4, 1, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    v, out2 = k.clone(), out.clone()
    bad, kv = i32([[0, 9, 9, 9]]), i32([64])
    for _ in range(20):
        for stream in (None, side):
            pc.gather(k, v, bad, kv, 0, out.view(1, 1, 1, 64, 128), out2.view(1, 1, 1, 64, 128), stream=stream)
            with pytest.raises(wi.WiError, match="page or slot"):
                pc.check()
    pc.check()
    pc.free()


def test_outputs_are_made_on_the_stream_that_a_handle_names(wi):
    """An output that a call makes itself belongs to the call's stream, given as an object or as a handle; 0 is the
    default stream, also while another one is current."""
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for stream, want in ((None, 0), (0, 0), (1, 0), (torch.cuda.default_stream(), 0), (side, side.cuda_stream),
                         (side.cuda_stream, side.cuda_stream)):
        made = []

        def make(shape, dtype, device):
            made.append(torch.cuda.current_stream().cuda_stream)
            return torch.empty(shape, dtype=dtype, device=device)

        wi._new_on(stream, (4,), torch.float32, torch.device(DEV), make)
        if stream is not None:
            with torch.cuda.stream(other):
                wi._new_on(stream, (4,), torch.float32, torch.device(DEV), make)
        assert made == [want] * len(made), (stream, made, want)
    rng = np.random.default_rng(52)
    table, n_pages = lay_out([700], 16, rng)
    q, k, v = (bf(rng.normal(size=s))[0] for s in ((40, 8, 128), (n_pages, 2, 16, 128), (n_pages, 2, 16, 128)))
    pc = wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, 1, table.shape[1]))
    args = (q, k, v, i32(table), i32([0, 30]), i32([700]))
    want = pc.attention(*args)
    for stream in (0, 1, side.cuda_stream):
        torch.cuda.synchronize()
        got = pc.attention(*args, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    pc.check()
    pc.free()


# ------------------------------------------------------------ refusals ----

def test_tables_refuse_more_tokens_than_a_step_may_have(wi):
    """The limit of a step is the same for the tables as for the calls that use them; nothing is written."""
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 8, 2, 4))
    most = 1 << 24
    one = lambda: i32([0])  # noqa: E731
    table, kv, start, left = i32([[-1] * 4]), one(), i32([5, 5]), one()
    free = i32(range(8))
    for n, error in ((most + 1, wi.WiError), ((1 << 31) - 1, wi.WiError), (1 << 31, ValueError)):
        slots, pos = (torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(2))
        slots[:40] = 7
        with pytest.raises(error, match="tokens"):
            pc.tables(one(), i32([20]), free, i32([8]), table, kv, start, slots, pos, left)
        assert (slots[:40] == 7).all() and (start == 5).all() and (table == -1).all()
        del slots, pos
    slots, pos = (torch.full((most,), 7, dtype=torch.int32, device=DEV) for _ in range(2))
    pc.tables(one(), i32([20]), free, i32([8]), table, kv, start, slots, pos, left)
    pc.check()
    assert table[0].tolist() == [7, 6, -1, -1] and start.tolist() == [0, 20] and left.tolist() == [6]
    assert slots[:20].tolist() == [7 * 16 + i for i in range(16)] + [6 * 16 + i for i in range(4)]
    assert (slots[20:] == -1).all() and (pos[20:] == -1).all() and pos[:20].tolist() == list(range(20))
    pc.free()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("start,good", [
    ([0, 5, 2, 5], 1),                  # request 2 alone would be fine, and write rows of request 0
    ([0, 5, 7, 3, 10, 12], 2),
    ([0, 12, 0, 12, 0, 12], 1),         # every other request claims all rows
    ([5, 4, 4, 12], 0),
    ([0, 3, 3, 12, 11], 3),
    ([0] + [6, 2] * 250, 1),            # in another thread's share of the requests
    ([0] * 450 + [7, 1, 9], 450),
])
def test_attention_keeps_requests_apart_where_offsets_fall(wi, start, good):
    """The requests in front of a falling offset are answered as if they were the whole call; rows of none behind it."""
    rng = np.random.default_rng(53)
    n, batch = 12, len(start) - 1
    table, n_pages = lay_out([300], 16, rng)
    q, k, v = (bf(rng.normal(size=s))[0] for s in ((n, 8, 128), (n_pages, 2, 16, 128), (n_pages, 2, 16, 128)))
    pc = wi.PagedCache(wi.make_paged_config(8, 2, 16, n_pages, max(batch, 1), table.shape[1]))
    table, kv = i32(table.repeat(batch, 0)), i32([300] * batch)
    outs, lses = ([torch.full(s, 7.0, dtype=t, device=DEV) for _ in range(2)]
                  for s, t in (((n, 8, 128), torch.bfloat16), ((n, 8), torch.float32)))
    if good:
        pc.attention(q, k, v, table, i32(start[:good + 1]), kv[:good].contiguous(), out=outs[0], lse=lses[0])
        pc.check()
    pc.attention(q, k, v, table, i32(start), kv, out=outs[1], lse=lses[1])
    with pytest.raises(wi.WiError, match="length"):
        pc.check()
    assert torch.equal(*outs) and torch.equal(*lses)
    assert (outs[1][start[good]:] == 7).all() and (outs[1][start[0]:start[good]] != 7).any(-1).all()
    pc.free()


# ------------------------------------------------------------ from pages to an index ----

@pytest.mark.parametrize("layers", [1, 3])
def test_index_from_the_pages_of_several_layers(wi, layers):
    """An index built from the pages decodes as one built from the same rows laid out by hand."""
    rng = np.random.default_rng(54 + layers)
    batch, hq, hkv, page, n = 2, 8, 2, 16, 1024
    kv = [1100, 1024]
    table, n_pages = lay_out(kv, page, rng)
    pools = [bf(rng.normal(size=(layers, n_pages, hkv, page, 128)))[0] for _ in range(2)]
    rows = [torch.stack([torch.stack([torch.cat([pool[a, int(table[b, j])] for j in range(n // page)], 1)
                                      for a in range(layers)]) for b in range(batch)]) for pool in pools]
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, page, n_pages, batch, table.shape[1]))
    cfg = wi.make_config(batch, layers, hq, hkv, n, seg_len=512, clusters_per_seg=32, iters=2, budget_k=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ix = wi.WaveIndex.build_paged(cfg, pc, *pools, i32(table), i32(kv), stream=side)
    torch.cuda.synchronize()
    pc.check()
    iy = wi.WaveIndex.build(cfg, *rows)
    q = bf(rng.normal(size=(batch, layers, hq, 128)))[0]
    a, b = ix.decode(q), iy.decode(q)
    assert torch.equal(a, b) and a.isfinite().all() and (a != 0).any()
    for x in (ix, iy):
        x.check()
        x.free()
    pc.free()


@pytest.mark.parametrize("kv", [[1024, 1023], [0, 1024], [-1, 1024], [1024, 3000]])
@pytest.mark.parametrize("on", ["current", "side"])
def test_index_from_pages_wants_every_position(wi, kv, on):
    """A prompt shorter than the index's context, or longer than its row of pages, is no index over zeros."""
    rng = np.random.default_rng(55)
    hkv, page, n = 2, 16, 1024
    table, n_pages = lay_out([1100, 1100], page, rng)
    pools = [bf(rng.normal(size=(n_pages, hkv, page, 128)))[0] for _ in range(2)]
    pc = wi.PagedCache(wi.make_paged_config(8, hkv, page, n_pages, 2, table.shape[1]))
    cfg = wi.make_config(2, 1, 8, hkv, n, seg_len=512, clusters_per_seg=32, iters=2, budget_k=8)
    lengths, late, table = i32([1024, 1024]), i32(kv), i32(table)
    stream = torch.cuda.Stream() if on == "side" else torch.cuda.current_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):      # the lengths come late, on the call's stream
        torch.cuda._sleep(20_000_000)
        lengths.copy_(late)
    short = next(b for b, x in enumerate(kv) if not n <= x <= table.shape[1] * page)
    with pytest.raises(ValueError, match=rf"kv_len\[{short}\].*got {kv[short]}"):
        wi.WaveIndex.build_paged(cfg, pc, *pools, table, lengths, stream=stream)
    torch.cuda.synchronize()
    pc.free()


# ------------------------------------------------------------ failed launches ----

@pytest.mark.parametrize("call", ["tables", "write", "attention", "gather"])
def test_a_launch_that_fails_leaves_nothing_behind(wi, call):
    """A call on the default stream while a stream that waits for it is captured cannot be launched: it says so, and the
    next call of the library, which has nothing to do with it, is fine."""
    import ctypes

    cu = ctypes.CDLL("libcuda.so.1")
    pc = wi.PagedCache(wi.make_paged_config(4, 2, 16, 8, 1, 4))
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    q, kn = torch.zeros((1, 4, 128), **bf16), torch.zeros((1, 2, 128), **bf16)
    vn, qo, out = kn.clone(), q.clone(), q.clone()
    pools = [torch.zeros((8, 2, 16, 128), **bf16) for _ in range(2)]
    rows = [torch.zeros((1, 1, 2, 4, 128), **bf16) for _ in range(2)]
    table, one, start = i32([[0, 1, 2, 3]]), [i32([1]) for _ in range(8)], i32([0, 1])
    free = i32([4, 5])
    cfg = wi.make_config(1, 1, 4, 2, 1024, seg_len=512, clusters_per_seg=32)
    keys = torch.zeros((1, 1, 2, 1024, 128), **bf16)
    mu = torch.zeros((2, 64, 128), **bf16)
    run = {"tables": lambda s: pc.tables(one[0], one[1], free, one[2], table, one[3], start, one[4], one[5], one[6], stream=s),
           "write": lambda s: pc.write(q, kn, vn, one[0], one[1], *pools, qo, stream=s),
           "attention": lambda s: pc.attention(q, *pools, table, start, one[0], out=out, stream=s),
           "gather": lambda s: pc.gather(*pools, table, one[0], 0, *rows, stream=s)}[call]
    run(None)
    wi.wi_init_centroids(cfg, keys, mu)
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
    wi.wi_init_centroids(cfg, keys, mu)
    run(None)
    pc.check()
    pc.free()


# ------------------------------------------------------------ angles of far positions ----

def test_write_knows_the_angles_of_far_positions(wi):
    """At position 2^31 - 1 and frequencies whose angle lies within 2e-6 of a quarter turn, (1, 0) turns to (+-2e-6 or
    less, +-1): the first element's bf16 digits show the angle to about 2^-30 of a turn.  The frequencies are such that
    their quotient by 2 pi, rounded to a double, would be off by 24 * 2^-32 of a turn there or more, while the angle's own
    rounding to fp32 is at most 1.5 * 2^-32."""
    from fractions import Fraction

    turn = Fraction(2 * 3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)
    rng = np.random.default_rng(56)
    p, freq, want = 2 ** 31 - 1, [], []
    while len(freq) < 64:
        k, quarter = int(rng.integers(1, p // 8)), int(rng.choice([-1, 1]))
        f = float((k * turn + quarter * turn / 4 + Fraction(rng.uniform(2e-7, 2e-6) * rng.choice([-1, 1]))) / p)
        exact = Fraction(f) * p / turn
        exact -= round(exact)                                    # turns in [-1/2, 1/2]
        units = int(np.floor(float(exact * 2 ** 32)))
        rounded = float(f / (2 * np.pi))
        near = Fraction(rounded) * p
        near -= round(near)
        if abs(int(np.float32(units)) - units) <= 1.5 and abs(near - exact) * 2 ** 32 >= 24:
            freq.append(f)
            want.append((float(np.cos(float(exact * turn))), quarter))
    want = np.array(want)
    x = torch.zeros((1, 3, 128), dtype=torch.bfloat16, device=DEV)
    x[..., :64] = 1
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 1, 1, 1, inv_freq=freq))
    pools = [torch.zeros((1, 1, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = f64(pc.write(x[:, :1], x[:, 1:2], x[:, 2:], i32([p]), i32([0]), *pools))[0, 0]
    pc.check()
    pc.free()
    # half a step of bf16, cosine and product in fp32 (2^-21 of the value), and of the angle: 1 for the product's dropped
    # bits, 1.5 for its rounding, 0.5 for the frequency, in 2^-32 turns
    tol = (2.0 ** -8 + 2.0 ** -21) * np.abs(want[:, 0]) + 3 * 2.0 ** -32 * 2 * np.pi
    assert (np.abs(out[:64] - want[:, 0]) <= tol).all(), (np.abs(out[:64] - want[:, 0]) / tol).max()
    assert (out[64:] == want[:, 1]).all()


def test_write_turns_backwards(wi):
    """Negative frequencies turn as positive ones mirrored, tiny ones (whose fraction of a turn is next to a whole) too."""
    rng = np.random.default_rng(57)
    n, freq = 40, [float(f) for f in 10.0 ** rng.uniform(-22, 0.7, size=64)]
    x = bf(rng.normal(size=(n, 3, 128)))[0]
    pos, slots = i32(rng.integers(0, 2 ** 31 - 1, n)), i32(range(n))
    got = []
    for sign in (1, -1):
        pc = wi.PagedCache(wi.make_paged_config(1, 1, 16, 3, 1, 1, inv_freq=[sign * f for f in freq]))
        pools = [torch.zeros((3, 1, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        y = x if sign > 0 else torch.cat([x[..., 64:], x[..., :64]], -1)      # (a, b) as (b, a): the other way round
        got.append(f64(pc.write(y[:, :1], y[:, 1:2], y[:, 2:], pos, slots, *pools)))
        pc.check()
        pc.free()
    a, b = got[0], np.concatenate([got[1][..., 64:], got[1][..., :64]], -1)
    size = np.abs(f64(x[:, :1]))
    size = np.concatenate([size[..., :64] + size[..., 64:]] * 2, -1)
    # each is off by half a step of bf16 and 2^-23 of |a| + |b| (angles of 2^-26 turns, products and sums in fp32)
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(a) + 2.0 ** -19 * size + 2.0 ** -133).all()


# ------------------------------------------------------------ contexts of millions of positions ----

def repeated(kv, rng, rows=1024):
    """Block table of a long request over a pool of few pages of 128, each position's row, and the rows' counts in front
    of positions [kv - tail, kv)."""
    table = rng.integers(0, rows // 128, -(-kv // 128))
    row = (table[:, None] * 128 + np.arange(128)).reshape(-1)[:kv]
    return table, row


@pytest.mark.parametrize("hq,hkv,new,kv", [
    (8, 2, [1] * 80, [1 << 20] * 80),                          # one tile, whole in their CTAs, segment after segment
    (4, 1, [1], [(1 << 26) - 77]),                             # cut: every CTA has more than a segment of it
    (4, 1, [40], [(1 << 26) - 77]),                            # two tiles, cut
    (4, 1, [40] * 200, [(1 << 19) + 300] * 200),               # two tiles, whole or cut anywhere
    (8, 1, [1, 33, 2, 0, 16, 1, 70], [1 << 23, 3 << 20, 900, 5, (1 << 22) + 1, 7 << 20, 555555]),
])
def test_attention_over_millions_of_positions(wi, hq, hkv, new, kv):
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
    (q, Q), (k, K), (v, V) = (bf(rng.normal(size=s)) for s in ((n, hq, 128), (8, hkv, 128, 128), (8, hkv, 128, 128)))
    pc = wi.PagedCache(wi.make_paged_config(hq, hkv, 128, 8, len(kv), width))
    lse = torch.empty((n, hq), device=DEV)
    args = (q, k, v, i32(table), i32(start), i32(kv))
    out = pc.attention(*args, lse=lse)
    pc.check()
    again = pc.attention(*args)
    pc.check()
    pc.free()
    assert torch.equal(out, again)
    out, lse = f64(out), f64(lse)
    K, V = (x.transpose(1, 0, 2, 3).reshape(hkv, -1, 128) for x in (K, V))
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
                # weights and result rounded to bf16, 2^-8 each; a score of at most 40 off by 128 * 2^-24 * 40 < 2^-11,
                # twice; a segment's 2^14 additions of sixteen positions' products, each in up to four steps that lose
                # less than 2^-23 of a sum that is half as large on average, 2^-8; its 2^11 sums of a row, less
                assert (np.abs(out[t, h] - ref) <= 2.0 ** -8 * np.abs(ref) + (3 * 2.0 ** -8) * spread).all()
                assert abs(lse[t, h] - (np.log(z) + x.max())) <= 2.0 ** -11 + 2.0 ** -12


def test_attention_adds_long_contexts_up_in_parts(wi):
    """Equal scores over values of one sign: what the additions lose does not grow with the context (in one sum, 2^23
    positions came out 2.2% too small).  A bf16 rounding, and the additions' 2^-8 as above."""
    rng = np.random.default_rng(59)
    kv, batch = 1 << 23, 2 * 152
    table, row = repeated(kv, rng)
    v, V = bf(rng.uniform(0.5, 1.5, size=(8, 1, 128, 128)))
    k = torch.zeros_like(v)
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 128, 8, batch, len(table)))
    q = torch.zeros((batch, 1, 128), dtype=torch.bfloat16, device=DEV)
    out = pc.attention(q, k, v, i32(table)[None].repeat(batch, 1), i32(range(batch + 1)), i32([kv] * batch))
    pc.check()
    pc.free()
    ref = np.bincount(row, minlength=1024) / kv @ V.reshape(1024, 128)
    assert (np.abs(f64(out) - ref) <= 2.0 ** -7 * ref).all()


@pytest.mark.parametrize("hq,new", [(1, 300), (4, 40)])
def test_attention_poison_where_a_long_context_is_cut(wi, hq, new):
    """Infinite and NaN values on both sides of position 2^18, where the first 2048 blocks end, in the middle of the
    tokens' own positions: they reach the tokens that see them, in their two elements, and no others."""
    rng = np.random.default_rng(60)
    kv, batch, at = (1 << 18) + new // 2, 100, ((1 << 18) - 9, (1 << 18) + 3)
    table, row = repeated(kv, rng)
    table[-4:] = [8, 9, 10, 11]                 # the last blocks' pages are used once
    row = (table[:, None] * 128 + np.arange(128)).reshape(-1)[:kv]
    K, V = rng.normal(size=(12, 1, 128, 128)), rng.normal(size=(12, 1, 128, 128))
    flat = V.reshape(-1, 128)
    flat[row[at[0]], 9], flat[row[at[1]], 70] = np.inf, np.nan
    (q, Q), (k, K), (v, V) = bf(rng.normal(size=(new, hq, 128))), bf(K), bf(V)
    pc = wi.PagedCache(wi.make_paged_config(hq, 1, 128, 12, batch, len(table)))
    out = pc.attention(q.repeat(batch, 1, 1), k, v, i32(table)[None].repeat(batch, 1), i32(np.arange(batch + 1) * new),
                       i32([kv] * batch))
    pc.check()
    pc.free()
    out = f64(out).reshape(batch, new, hq, 128)
    K, V = K.reshape(-1, 128), V.reshape(-1, 128)
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
            assert (got[..., 9] == np.inf).all(), i
        if p >= at[1]:
            assert np.isnan(got[..., 70]).all(), i
        fine = np.ones(128, bool)
        fine[[9] * (p >= at[0]) + [70] * (p >= at[1])] = False
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -8 * spread)[..., fine].all(), i

def test_attention_over_a_quarter_of_a_billion_positions(wi):
    """Two million blocks of one item in a CTA, nearly three seconds: longer than a wait is given.  One page holds every
    position; with equal scores and powers of two as values every sum is exact."""
    kv, n = 1 << 28, 256 * torch.cuda.get_device_properties(0).multi_processor_count
    pc = wi.PagedCache(wi.make_paged_config(1, 1, 128, 1, 1, kv // 128))
    k = torch.zeros((1, 1, 128, 128), dtype=torch.bfloat16, device=DEV)
    v = bf(np.broadcast_to(2.0 ** (np.arange(128) % 4), k.shape))[0]
    q = torch.zeros((n, 1, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((n, 1), device=DEV)
    out = pc.attention(q, k, v, torch.zeros((1, kv // 128), dtype=torch.int32, device=DEV), i32([0, n]), i32([kv]), lse=lse)
    pc.check()
    pc.free()
    assert (out == v[0, 0, 0]).all()
    assert (lse - 28 * np.log(2)).abs().max() < 2.0 ** -12       # the rows see 2^28 positions and up to n fewer
