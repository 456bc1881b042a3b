"""Cases that measure the paged cache in 8 bits and rotations by positions of several axes: the write of normed and
rotated queries and keys (bf16 pools, positions of time, height and width), the write that appends keys and values to
8-bit pools, attention over those, and the gather of their rows into the layout that the wave index is built from.

An 8-bit pool holds e4m3 values [page][kv head][position][128] and a power of two [page][kv head][position / 16] for
every sixteen positions of a head, by which the values are multiplied; rows are otherwise those of the bf16 pools.
"""
import math
import random

import torch

own = False

D = 128
GROUP = 16         # positions that share a scale
TOP = 448.0        # the largest e4m3 value
LOWEST = -64       # the smallest exponent of a scale
THETA = 500000.0   # the rotation base of this repository's workloads
EPS = 1e-6
SPARE = 7          # pages of a pool that no request holds

HEADS = [(32, 8), (28, 4), (8, 1), (4, 4), (6, 2), (5, 1), (12, 4), (6, 1), (16, 8), (1, 1)]
PAGES = [16, 16, 32, 48, 64, 128, 256]


def listed():
    def case(name, op, **kw):
        return dict(name=name, op=op, **kw)

    return [
        # the tokens of one small picture after a few words, 28 query and 4 kv heads: latency
        case("axes_picture_70", "axes", tokens=70, hq=28, hkv=4, page=16, rotary=128, interleaved=False, norm=True, pad=2),
        # a prefill chunk of video frames, one segment of the index long
        case("axes_video_8192", "axes", tokens=8192, hq=32, hkv=8, page=64, rotary=128, interleaved=False, norm=True, pad=0),
        # one token of each of sixteen requests (the batch of the 120K workload), most of them inside a group of sixteen
        case("write8_decode_16", "write8", batch=16, q_lo=1, q_hi=1, ctx_lo=100, ctx_hi=9000, lens=11, hq=32, hkv=8, page=16,
             rotary=128, interleaved=False, norm=True, axes=1, pad=0),
        # odd chunks of five requests in a padded buffer, half of each head rotated by three axes, the Qwen-shaped heads
        case("write8_odd_5", "write8", batch=5, q_lo=1, q_hi=600, ctx_lo=0, ctx_hi=700, lens=12, hq=28, hkv=4, page=48,
             rotary=64, interleaved=True, norm=True, axes=3, pad=5),
        # a prefill chunk of one segment of the index
        case("write8_chunk_8192", "write8", batch=1, q_lo=8192, q_hi=8192, ctx_lo=8192, ctx_hi=8192, lens=0, hq=32, hkv=8,
             page=64, rotary=128, interleaved=False, norm=True, axes=1, pad=0),
        # a follow-up of a few tokens in a short conversation: latency
        case("attn8_short_5", "attention8", batch=1, hq=32, hkv=8, page=16, q_lo=5, q_hi=5, ctx_lo=300, ctx_hi=300, pad=0,
             lens=0),
        # single tokens of many requests of ragged length: a serving batch
        case("attn8_batch_64", "attention8", batch=64, hq=32, hkv=8, page=16, q_lo=1, q_hi=1, ctx_lo=100, ctx_hi=8000, pad=0,
             lens=14),
        # one token over the 131K context of this repository's headline decode workload
        case("attn8_decode_131k", "attention8", batch=1, hq=32, hkv=8, page=16, q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071,
             pad=0, lens=0),
        # chunks and single tokens of seven requests in one call, odd lengths, seven query heads to a kv head
        case("attn8_mixed_7", "attention8", batch=7, hq=28, hkv=4, page=64, q_lo=1, q_hi=777, ctx_lo=0, ctx_hi=9000, pad=3,
             lens=4),
        # a prefill chunk deep in a 131K prompt
        case("attn8_chunk_131k", "attention8", batch=1, hq=32, hkv=8, page=128, q_lo=2048, q_hi=2048, ctx_lo=129024,
             ctx_hi=129024, pad=0, lens=0),
        # the row that each request appends to its index
        case("gather8_append_16", "gather8", batch=16, layers=1, hkv=8, page=16, rows=1, kv_lo=5000, kv_hi=8000, lens=5),
        # a whole 131K prompt into the layout of the index build
        case("gather8_131k", "gather8", batch=1, layers=1, hkv=8, page=16, rows=131072, kv_lo=131072, kv_hi=131072, lens=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["axes", "write8", "write8", "attention8", "attention8", "gather8"])
    page, lens = rng.choice(PAGES), rng.randrange(1, 1 << 20)
    hq, hkv = rng.choice(HEADS)
    turn = dict(rotary=rng.choice([32, 64, 96, 128]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.7)
    if op == "axes":
        return dict(op=op, tokens=_log(rng, 1, 8000), hq=hq, hkv=hkv, page=page,
                    pad=rng.choice([0, rng.randrange(1, 40)]), **turn)
    if op == "write8":
        batch = _log(rng, 1, 64)
        q_hi = _log(rng, 1, 8000 // batch)
        return dict(op=op, batch=batch, q_lo=rng.choice([1, q_hi]), q_hi=q_hi, ctx_lo=0, ctx_hi=_log(rng, 1, 16000 // batch),
                    lens=lens, hq=hq, hkv=hkv, page=page, axes=rng.choice([1, 1, 3]),
                    pad=rng.choice([0, rng.randrange(1, 40)]), **turn)
    if op == "gather8":
        batch, layers = rng.choice([1, 1, 2, 3, 5]), rng.choice([1, 1, 2, 3])
        kv_hi = _log(rng, 2, 1000000 // (batch * layers * hkv))
        return dict(op=op, batch=batch, layers=layers, hkv=hkv, page=page, rows=rng.choice([1, _log(rng, 1, kv_hi)]),
                    kv_lo=max(1, kv_hi // 2), kv_hi=kv_hi, lens=lens)
    kind = rng.choice(["single", "chunk", "mixed"])
    if kind == "single":
        batch = _log(rng, 1, 64)
        ctx_hi = _log(rng, 1, 131000 // batch)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, page=page, q_lo=1, q_hi=1, ctx_lo=ctx_hi // 3, ctx_hi=ctx_hi,
                    pad=0, lens=lens)
    batch = 1 if kind == "chunk" else rng.randrange(2, 12)
    q_hi = _log(rng, 2, 2000 if kind == "chunk" else 900)
    ctx_hi = _log(rng, 1, min(120000 // batch, (1 << 28) // (q_hi * batch)))
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, page=page, q_lo=q_hi if kind == "chunk" else 1, q_hi=q_hi, ctx_lo=0,
                ctx_hi=ctx_hi, pad=rng.choice([0, 9]), lens=lens)


# ---------------------------------------------------------------- the inputs ----

def _lengths(case):
    """(context before the step, new tokens) of every request: part of the case, the same for every seed."""
    r = random.Random(case["lens"] * 7919 + 13)

    def one(lo, hi):
        return lo if r.random() < 0.3 else r.randint(lo, hi)

    ctx = [one(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [one(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    return ctx, new


def _kv_lengths(case):
    r = random.Random(case["lens"] * 7919 + 13)
    return [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["batch"])]


def _up(a, b):
    return -(-a // b)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _inv_freq(rotary):
    return [THETA ** (-2.0 * i / rotary) for i in range(rotary // 2)]


def _axis_of(rotary):
    """The axis (time, height, width) of every pair: a quarter of them time, the rest height and width by turns."""
    pairs = rotary // 2
    return [0 if i < pairs // 4 else 1 + i % 2 for i in range(pairs)]


def _pool(n_pages, hkv, page, gen, layers=None):
    """Rows of a bf16 cache: a common direction that the heads' keys share and noise of unit size on it."""
    shape = ((layers,) if layers else ()) + (n_pages, hkv, page, D)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return x.add_(torch.randn((hkv, 1, D), generator=gen, device="cuda", dtype=torch.bfloat16), alpha=0.5)


def _scale_of(top):
    """The exponent e of the smallest power of two with top <= 448 * 2^e."""
    m, x = torch.frexp(top)
    return torch.where(top > 0, x - 9 + (m > 0.875), LOWEST).clamp(min=LOWEST)


def _as_scales(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _exponents(scales):
    return scales.view(torch.uint8).int() - 127


def _pool8(n_pages, hkv, page, gen, layers=None):
    """The same rows, their size changing a little from group to group, held in 8 bits: values and scales."""
    x = _pool(n_pages, hkv, page, gen, layers).unflatten(-2, (page // GROUP, GROUP))
    size = torch.randn(x.shape[:-2] + (1, 1), generator=gen, device="cuda").mul_(0.3).exp_()
    x = x * size.bfloat16()
    e = _scale_of(x.abs().amax((-1, -2)).float())
    x = (x * torch.exp2(-e.float())[..., None, None].bfloat16()).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
    return x.flatten(-3, -2), _as_scales(e)


def _table(kv, page, gen):
    """Block table (rows padded with -1) with the requests' pages scattered over the pool, and the pool's size."""
    used = [_up(n, page) for n in kv]
    n_pages = sum(used) + SPARE
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(kv), max(max(used), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _cache(case, n_pages, max_pages, hq, axes=None, **kw):
    """The handle that a user's program keeps for its paged cache."""
    if not own:
        return None
    import clustered_sparse_kv_gb300 as wi

    return wi.PagedCache(wi.make_paged_config(hq, case.get("hkv", 1), case["page"], n_pages,
                                              max_batch=case.get("batch", 1), max_pages=max_pages, **kw), axes=axes)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"op": case["op"], "case": case}
    page = case["page"]
    if case["op"] in ("axes", "write8"):
        hq, hkv, rotary = case["hq"], case["hkv"], case["rotary"]
        if case["op"] == "axes":
            axes, live = 3, case["tokens"]
            n_pages = _up(live, page) + SPARE
            slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:live]
            s.update(k_pages=_pool(n_pages, hkv, page, gen), v_pages=_pool(n_pages, hkv, page, gen))
        else:
            axes = case["axes"]
            ctx, new = _lengths(case)
            live = sum(new)
            table, n_pages = _table([c + n for c, n in zip(ctx, new)], page, gen)
            b = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(new, device="cuda"))
            starts = torch.tensor([sum(new[:i]) for i in range(len(new))], device="cuda")
            at = torch.tensor(ctx, device="cuda")[b] + torch.arange(live, device="cuda") - starts[b]
            slots = table[b, at // page].long() * page + at % page
            for name in ("k", "v"):
                s[name + "_pages"], s[name + "_scales"] = _pool8(n_pages, hkv, page, gen)
        n = live + case["pad"]
        slots = torch.cat([slots.int(), _ints([-1] * case["pad"])])
        if axes == 1:
            positions = torch.cat([at.int(), _ints([-1] * case["pad"])])
        else:  # time counts on; height and width are places in a picture
            positions = torch.randint(0, 400, (axes, n), generator=gen, device="cuda", dtype=torch.int32)
            positions[0] = torch.arange(n, device="cuda", dtype=torch.int32) // 64 + 40
            positions[:, live:] = -1
        weights = [(1 + 0.2 * torch.randn((D,), generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2)]
        freq, axis = _inv_freq(rotary), _axis_of(rotary) if axes > 1 else None
        s.update(qkv=torch.randn((n, (hq + 2 * hkv) * D), generator=gen, device="cuda", dtype=torch.bfloat16),
                 slots=slots, positions=positions, live=live, q_weight=weights[0] if case["norm"] else None,
                 k_weight=weights[1] if case["norm"] else None,
                 q_out=torch.zeros((n, hq, D), device="cuda", dtype=torch.bfloat16),
                 inv_freq=torch.tensor(freq, dtype=torch.float64, device="cuda"),
                 axis=torch.tensor(axis or [0] * (rotary // 2), device="cuda"),
                 cache=_cache(case, n_pages, 1, hq, axes=axis, rotary_dim=rotary, interleaved=case["interleaved"],
                              inv_freq=freq, eps=EPS))
    elif case["op"] == "attention8":
        ctx, new = _lengths(case)
        kv = [c + n for c, n in zip(ctx, new)]
        table, n_pages = _table(kv, page, gen)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        n = starts[-1] + case["pad"]
        q = torch.randn((n, case["hq"], D), generator=gen, device="cuda", dtype=torch.bfloat16) * 1.5
        for name in ("k", "v"):
            s[name + "_pages"], s[name + "_scales"] = _pool8(n_pages, case["hkv"], page, gen)
        s.update(q=q, block_table=table, q_start=_ints(starts), kv_len=_ints(kv), out=torch.zeros_like(q),
                 lse=torch.zeros((n, case["hq"]), device="cuda"), max_q=max(new), max_kv=max(kv),
                 cache=_cache(case, n_pages, table.shape[1], case["hq"]))
    else:
        kv = _kv_lengths(case)
        table, n_pages = _table(kv, page, gen)
        shape = (case["batch"], case["layers"], case["hkv"], case["rows"], D)
        for name in ("k", "v"):
            s[name + "_pages"], s[name + "_scales"] = _pool8(n_pages, case["hkv"], page, gen, case["layers"])
        s.update(block_table=table, kv_len=_ints(kv), pos0=min(kv) - min(min(kv), case["rows"]),
                 k_out=torch.zeros(shape, device="cuda", dtype=torch.bfloat16),
                 v_out=torch.zeros(shape, device="cuda", dtype=torch.bfloat16),
                 cache=_cache(case, n_pages, table.shape[1], case["hkv"]))
    return s


# ------------------------------------------------------------- one pass ----

def run(state):
    return {"axes": _axes, "write8": _write8, "attention8": _attention8, "gather8": _gather8}[state["op"]](state)


def _parts(s):
    hq, hkv, n = s["case"]["hq"], s["case"]["hkv"], s["qkv"].shape[0]
    q, k, v = s["qkv"].split([hq * D, hkv * D, hkv * D], 1)
    return q.view(n, hq, D), k.view(n, hkv, D), v.view(n, hkv, D)


def _turned(s, x, weight):
    """x normed and rotated, in 32 bits (angles in 64)."""
    c, live = s["case"], s["live"]
    rotary, inter = c["rotary"], c["interleaved"]
    x = x[:live].float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    positions = s["positions"].reshape(-1, s["qkv"].shape[0])[s["axis"], :live]   # [pair, token]
    angle = (positions.double() * s["inv_freq"][:, None]).T[:, None]
    cos, sin = angle.cos().float(), angle.sin().float()
    part, rest = x[..., :rotary], x[..., rotary:]
    a, b = (part[..., 0::2], part[..., 1::2]) if inter else (part[..., :rotary // 2], part[..., rotary // 2:])
    pair = [a * cos - b * sin, b * cos + a * sin]
    part = torch.stack(pair, -1).flatten(-2) if inter else torch.cat(pair, -1)
    return torch.cat([part, rest], -1)


def _axes(s):
    q, k, v = _parts(s)
    if own:
        s["cache"].write(q, k, v, s["positions"], s["slots"], s["k_pages"], s["v_pages"], s["q_out"],
                         q_weight=s["q_weight"], k_weight=s["k_weight"])
    else:
        page, live = s["case"]["page"], s["live"]
        slots = s["slots"][:live].long()
        at, off = slots // page, slots % page
        s["q_out"][:live] = _turned(s, q, s["q_weight"]).bfloat16()
        s["k_pages"][at, :, off] = _turned(s, k, s["k_weight"]).bfloat16()
        s["v_pages"][at, :, off] = v[:live]
    return {k: s[k] for k in ("q_out", "k_pages", "v_pages")}


def _write8(s):
    q, k, v = _parts(s)
    names = ("q_out", "k_pages", "v_pages", "k_scales", "v_scales")
    if own:
        s["cache"].write8(q, k, v, s["positions"], s["slots"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                          s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"])
        return {k: s[k] for k in names}
    live = s["live"]
    s["q_out"][:live] = _turned(s, q, s["q_weight"]).bfloat16()
    _append(s, "k", _turned(s, k, s["k_weight"]))
    _append(s, "v", v[:live].float())
    return {k: s[k] for k in names}


def _append(s, name, x):
    """The rows x [token][kv head][128] into the slots of an 8-bit pool: a group's scale grows with its largest value,
    the rows that it held before are rounded again where it did; a group's first row begins it anew."""
    pages, scales, page = s[name + "_pages"].view(torch.uint8), s[name + "_scales"].view(torch.uint8), s["case"]["page"]
    slots = s["slots"][:s["live"]].long()
    group, of = (slots // GROUP).unique(return_inverse=True)      # the groups that the step touches, each token's
    off, hkv = slots % GROUP, x.shape[1]
    need = torch.full((len(group), hkv), LOWEST, dtype=torch.int32, device="cuda")
    need.scatter_reduce_(0, of[:, None].expand(-1, hkv), _scale_of(x.abs().amax(-1)).int(), "amax")
    first = torch.full((len(group),), GROUP, device="cuda").scatter_reduce_(0, of, off, "amin")
    at, sub = group // (page // GROUP), group % (page // GROUP)   # page of a group, place in the page
    was = scales[at, :, sub].int() - 127
    now = torch.where((first == 0)[:, None], need, torch.maximum(was, need))
    rows = pages.unflatten(2, (-1, GROUP))[at, :, sub]            # [group, kv head, row, 128]
    held = (torch.arange(GROUP, device="cuda") < first[:, None])[:, None] & (now > was)[..., None]
    again = rows.view(torch.float8_e4m3fn).float() * torch.exp2((was - now).float())[..., None, None]
    rows = torch.where(held[..., None], again.to(torch.float8_e4m3fn).view(torch.uint8), rows)
    x = (x * torch.exp2(-now[of].float())[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    rows[of, :, off] = x.view(torch.uint8)
    pages.unflatten(2, (-1, GROUP))[at, :, sub] = rows
    scales[at, :, sub] = (now + 127).to(torch.uint8)


def _attention8(s):
    if own:
        s["cache"].attention8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["block_table"],
                              s["q_start"], s["kv_len"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    c, kv = s["case"], s["kv_len"].long()
    hkv, g, page, start = c["hkv"], c["hq"] // c["hkv"], c["page"], s["q_start"].long()
    new = start[1:] - start[:-1]
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_kv"], device="cuda")
    live = i < new[:, None]                                       # [request, its token]
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    pages, off = s["block_table"][:, j // page].long().clamp(min=0), j % page
    seen = j <= (kv - new)[:, None, None] + i[:, None]            # [request, token, position]
    held = (j < kv[:, None])[..., None]
    q = s["q"].view(-1, hkv, g, D)

    def values(name, h):
        x = s[name + "_pages"].view(torch.uint8)[pages, h, off].view(torch.float8_e4m3fn).float()
        return x * torch.exp2(_exponents(s[name + "_scales"])[pages, h, off // GROUP].float())[..., None]

    for h in range(hkv):  # one kv head's score matrix at a time is what the memory holds
        k, v = values("k", h), torch.where(held, values("v", h), 0.0)
        x = torch.matmul(q[row, h].float().flatten(1, 2), k.transpose(1, 2)) * D ** -0.5
        x = x.unflatten(1, (s["max_q"], g)).masked_fill_(~seen[:, :, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        x = x.sub_(top).exp_()
        z = x.sum(-1, keepdim=True)
        y = torch.matmul(x.flatten(1, 2), v).unflatten(1, (s["max_q"], g)) / torch.where(z == 0, 1.0, z)
        s["out"].view(-1, hkv, g, D)[row[live], h] = y[live].bfloat16()
        s["lse"].view(-1, hkv, g)[row[live], h] = (top + z.log())[live].squeeze(-1)
    return {"out": s["out"], "lse": s["lse"]}


def _gather8(s):
    if own:
        s["cache"].gather8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["block_table"], s["kv_len"],
                           s["pos0"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    page = s["case"]["page"]
    j = s["pos0"] + torch.arange(s["case"]["rows"], device="cuda")
    pages, off = s["block_table"][:, (j // page).clamp(max=s["block_table"].shape[1] - 1)].long().clamp(min=0), j % page
    held = (j < s["kv_len"][:, None])[..., None, None, None]
    for name, to in (("k", s["k_out"]), ("v", s["v_out"])):
        # [layer, page, kv head, ...] -> [request, position, layer, kv head, ...]
        x = s[name + "_pages"].view(torch.uint8).permute(1, 3, 0, 2, 4)[pages, off].view(torch.float8_e4m3fn).float()
        e = _exponents(s[name + "_scales"]).permute(1, 3, 0, 2)[pages, off // GROUP].float()
        to.copy_(torch.where(held, x * torch.exp2(e)[..., None], 0.0).permute(0, 2, 3, 1, 4))
    return {"k": s["k_out"], "v": s["v_out"]}


# ------------------------------------------------------------- what it takes ----

def work(case):
    if case["op"] in ("axes", "write8"):
        hq, hkv, norm = case["hq"], case["hkv"], 4 if case["norm"] else 0
        tokens, axes, out = case.get("tokens"), 3, 2 * 2 * hkv * D
        more = 0
        if case["op"] == "write8":
            ctx, new = _lengths(case)
            tokens, axes, out = sum(new), case["axes"], 2 * hkv * D
            # scales: one of each group that the step touches, read where it was begun before
            more = sum(2 * hkv * (_up(c + n, GROUP) - c // GROUP + (c % GROUP > 0)) for c, n in zip(ctx, new))
        return {"bytes": tokens * ((hq + 2 * hkv) * 2 * D + hq * 2 * D + out + 4 + 4 * axes) + more
                + (4 * D if norm else 0) + 4 * case["rotary"],
                "flops": tokens * ((hq + hkv) * (norm * D + 3 * case["rotary"] + D) + (2 * hkv * 2 * D if more else 0))}
    if case["op"] == "attention8":
        ctx, new = _lengths(case)
        rows = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
        kv = [c + n for c, n in zip(ctx, new)]
        return {"bytes": sum(new) * case["hq"] * (4 * D + 4) + case["hkv"] * sum(2 * D * n + 2 * _up(n, GROUP) for n in kv)
                + 4 * sum(_up(n, case["page"]) for n in kv) + 8 * len(ctx) + 4,
                "flops": 4 * D * case["hq"] * rows}
    rows = case["batch"] * case["layers"] * case["hkv"] * case["rows"]
    return {"bytes": 6 * D * rows + 2 * _up(rows, GROUP) + 4 * case["batch"] * (1 + _up(case["rows"], case["page"])),
            "flops": 2 * D * rows}


# ------------------------------------------------------ from the definitions ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"axes": _exact_axes, "write8": _exact_write8, "attention8": _exact_attention8, "gather8": _exact_gather8}[
        case["op"]](s)


def _exact_heads(s):
    """q, k (normed and turned) and v of the live tokens."""
    c = s["case"]
    hq, hkv, rot, live = c["hq"], c["hkv"], c["rotary"], s["live"]
    heads = s["qkv"][:live].double().view(live, hq + 2 * hkv, D)
    # the pairs that turn together, and each pair's angle as a complex factor
    first = torch.arange(rot // 2, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else rot // 2)
    positions = s["positions"].double() if s["positions"].dim() == 2 else s["positions"].double()[None]
    angle = torch.stack([positions[a, :live] * f for a, f in zip(s["axis"].tolist(), s["inv_freq"])], 1)
    factor = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turn(x, weight):
        if weight is not None:
            x = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
        z = torch.complex(x[..., first], x[..., second]) * factor
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    return turn(heads[:, :hq], s["q_weight"]), turn(heads[:, hq:hq + hkv], s["k_weight"]), heads[:, hq + hkv:]


def _exact_axes(s):
    q, k, v = _exact_heads(s)
    got = {"q_out": s["q_out"].double(), "k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double()}
    got["q_out"][:s["live"]] = q
    page, slots = s["case"]["page"], s["slots"][:s["live"]].long()
    for name, x in (("k_pages", k), ("v_pages", v)):
        flat = got[name].transpose(1, 2).flatten(0, 1).clone()
        flat[slots] = x
        got[name] = flat.unflatten(0, (-1, page)).transpose(1, 2)
    return got


def _exact_write8(s):
    """The pools' values here are not rounded: what they stand for, over their group's scale."""
    q, k, v = _exact_heads(s)
    page, slots = s["case"]["page"], s["slots"][:s["live"]].cpu().long()
    got = {"q_out": s["q_out"].double()}
    got["q_out"][:s["live"]] = q
    begin = {}
    for g, o in zip((slots // GROUP).tolist(), (slots % GROUP).tolist()):
        begin[g] = min(o, begin.get(g, GROUP))
    touched = torch.tensor(list(begin), device="cuda")
    held = torch.arange(GROUP, device="cuda") < torch.tensor(list(begin.values()), device="cuda")[:, None]
    for name, x in (("k", k), ("v", v)):
        rows = s[name + "_pages"].double().transpose(1, 2).flatten(0, 1)          # [slot, kv head, 128]
        size = torch.exp2(_exponents(s[name + "_scales"]).double())
        size = size.transpose(1, 2).flatten(0, 1)                                 # [group, kv head]
        fresh = torch.zeros_like(rows)
        fresh[slots.cuda()] = x
        top = fresh.unflatten(0, (-1, GROUP))[touched].abs().amax((1, 3))
        want = torch.exp2(torch.ceil(torch.log2(top / TOP)).clamp(min=LOWEST))
        old = size[touched]
        new = torch.where(held[:, :1], torch.maximum(old, want), want)
        ratio = torch.ones_like(rows).unflatten(0, (-1, GROUP))
        ratio[touched] = torch.where(held[..., None, None], (old / new)[:, None, :, None], 1.0)
        rows = rows * ratio.flatten(0, 1)
        size = size.clone()
        size[touched] = new
        rows[slots.cuda()] = x / size[slots.cuda() // GROUP][..., None]
        got[name + "_pages"] = rows.unflatten(0, (-1, page)).transpose(1, 2)
        got[name + "_scales"] = size.unflatten(0, (-1, page // GROUP)).transpose(1, 2)
    return got


def _exact_rows(s, name, pages, layer=None):
    """The rows of these pages [..., kv head, position, 128] in 64 bits."""
    x, e = s[name + "_pages"], s[name + "_scales"]
    x, e = (x, e) if layer is None else (x[layer], e[layer])
    x, e = x.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double(), _exponents(e)[pages]
    return (x * torch.exp2(e.double()).repeat_interleave(GROUP, -1)[..., None]).transpose(0, 1).flatten(1, 2)


def _exact_attention8(s):
    c = s["case"]
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    ctx, new = _lengths(c)
    out, lse = s["out"].double(), s["lse"].double()
    at = 0
    for b in range(c["batch"]):
        n, kv = new[b], ctx[b] + new[b]
        pages = s["block_table"][b, :_up(kv, page)].long()
        ks, vs = _exact_rows(s, "k", pages), _exact_rows(s, "v", pages)
        for h in range(hq):
            k, v = ks[h // (hq // hkv), :kv], vs[h // (hq // hkv), :kv]
            x = s["q"][at:at + n, h].double() @ k.T / math.sqrt(D)
            x[:, ctx[b]:] += torch.full((n, n), -math.inf, dtype=torch.float64, device="cuda").triu(1)
            z = torch.logsumexp(x, 1)
            lse[at:at + n, h] = z
            out[at:at + n, h] = x.sub_(z[:, None]).exp_() @ v
        at += n
    return {"out": out, "lse": lse}


def _exact_gather8(s):
    c, page = s["case"], s["case"]["page"]
    got = {}
    for name in ("k", "v"):
        x = torch.zeros_like(s[name + "_out"], dtype=torch.float64)
        for b, kv in enumerate(_kv_lengths(c)):
            pages = s["block_table"][b, :_up(kv, page)].long()
            n = min(c["rows"], kv - s["pos0"])
            for layer in range(c["layers"]):
                x[b, layer, :, :n] = _exact_rows(s, name, pages, layer)[:, s["pos0"]:s["pos0"] + n]
        got[name] = x
    return got
