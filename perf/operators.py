"""Cases that measure the paged-cache operators: page tables from request lengths, per-head norms with the
position rotation written into the cache, attention of new tokens over it, and the gather of its rows into the
layout that the wave index is built from.

Head size 128 and bf16 rows throughout, as everywhere in this package; a page holds `page` positions of every
kv head, [kv head][position][128], and a request's pages are listed in its row of the block table.
"""
import math
import random

import torch

own = False

D = 128
THETA = 500000.0   # the rotation base of this repository's workloads
EPS = 1e-6
SPARE = 7          # pages of a pool that no request holds

HEADS = [(32, 8), (28, 4), (8, 1), (4, 4), (6, 2), (5, 1), (12, 4), (6, 1), (16, 8), (1, 1)]
PAGES = [16, 16, 32, 48, 64, 128, 256]


def listed():
    def tables(name, **kw):
        return dict(name=name, op="tables", **kw)

    def write(name, **kw):
        return dict(name=name, op="write", **kw)

    def attention(name, **kw):
        return dict(name=name, op="attention", **kw)

    def gather(name, **kw):
        return dict(name=name, op="gather", **kw)

    return [
        # one decode step of eight long requests: a launch's latency and little else
        tables("tables_decode_8", batch=8, page=16, q_lo=1, q_hi=1, ctx_lo=4000, ctx_hi=131071, pad=0, lens=1),
        # a serving step that mixes single tokens with chunks, in a token buffer of fixed size
        tables("tables_mixed_256", batch=256, page=64, q_lo=1, q_hi=300, ctx_lo=0, ctx_hi=20000, pad=517, lens=2),
        # first chunks of many requests at once: the largest maps
        tables("tables_prefill_64", batch=64, page=16, q_lo=1500, q_hi=4096, ctx_lo=0, ctx_hi=0, pad=0, lens=3),
        # one token of each of sixteen requests (the batch of the 120K workload)
        write("write_decode_16", tokens=16, hq=32, hkv=8, page=16, rotary=128, interleaved=False, norm=True, pad=0),
        # an odd chunk in a padded buffer, half of each head rotated, the Qwen-shaped heads
        write("write_odd_1531", tokens=1531, hq=28, hkv=4, page=48, rotary=64, interleaved=True, norm=True, pad=5),
        # a prefill chunk of one segment of the index
        write("write_chunk_8192", tokens=8192, hq=32, hkv=8, page=64, rotary=128, interleaved=False, norm=True, pad=0),
        # a follow-up of a few tokens in a short conversation: latency
        attention("attn_short_5", batch=1, hq=32, hkv=8, page=16, q_lo=5, q_hi=5, ctx_lo=300, ctx_hi=300, pad=0, lens=0),
        # one token over the 131K context of this repository's headline decode workload
        attention("attn_decode_131k", batch=1, hq=32, hkv=8, page=16, q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071,
                  pad=0, lens=0),
        # chunks and single tokens of seven requests in one call, odd lengths, seven query heads to a kv head
        attention("attn_mixed_7", batch=7, hq=28, hkv=4, page=64, q_lo=1, q_hi=777, ctx_lo=0, ctx_hi=9000, pad=3, lens=4),
        # a prefill chunk deep in a 131K prompt
        attention("attn_chunk_131k", batch=1, hq=32, hkv=8, page=128, q_lo=2048, q_hi=2048, ctx_lo=129024,
                  ctx_hi=129024, pad=0, lens=0),
        # the row that each request appends to its index
        gather("gather_append_16", batch=16, layers=1, hkv=8, page=16, rows=1, kv_lo=5000, kv_hi=8000, lens=5),
        # a whole 131K prompt into the layout of the index build
        gather("gather_131k", batch=1, layers=1, hkv=8, page=16, rows=131072, kv_lo=131072, kv_hi=131072, lens=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tables", "write", "attention", "attention", "gather"])
    page, lens = rng.choice(PAGES), rng.randrange(1, 1 << 20)
    hq, hkv = rng.choice(HEADS)
    if op == "tables":
        batch = _log(rng, 1, 900)
        q_hi = _log(rng, 1, max(1, 130000 // batch))
        ctx_hi = _log(rng, 1, 131072)
        return dict(op=op, batch=batch, page=page, q_lo=rng.choice([0, 1]), q_hi=q_hi, ctx_lo=0, ctx_hi=ctx_hi,
                    pad=rng.choice([0, _log(rng, 1, 600)]), lens=lens)
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 8000), hq=hq, hkv=hkv, page=page, rotary=rng.choice([0, 32, 64, 96, 128]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7, pad=rng.choice([0, rng.randrange(1, 40)]))
    if op == "gather":
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
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, page=page, q_lo=q_hi if kind == "chunk" else 1, q_hi=q_hi,
                ctx_lo=0, ctx_hi=ctx_hi, pad=rng.choice([0, 9]), lens=lens)


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


def _pool(n_pages, hkv, page, gen, layers=None):
    """Rows of a cache: a common direction that the heads' keys share and noise of unit size on it."""
    shape = ((layers,) if layers else ()) + (n_pages, hkv, page, D)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return x.add_(torch.randn((hkv, 1, D), generator=gen, device="cuda", dtype=torch.bfloat16), alpha=0.5)


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


def _cache(case, n_pages, max_pages, hq, **kw):
    """The handle that a user's program keeps for its paged cache."""
    if not own:
        return None
    import clustered_sparse_kv_gb300 as wi

    return wi.PagedCache(wi.make_paged_config(hq, case.get("hkv", 1), case["page"], n_pages,
                                              max_batch=case.get("batch", 1), max_pages=max_pages, **kw))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"op": case["op"], "case": case}
    page = case["page"]
    if case["op"] == "tables":
        ctx, new = _lengths(case)
        kv = [c + n for c, n in zip(ctx, new)]
        width = max(max(_up(n, page) for n in kv), 1) + 2
        held = [_up(c, page) for c in ctx]
        fresh = sum(_up(n, page) - h for n, h in zip(kv, held))
        n_pages = sum(held) + fresh + SPARE
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((len(kv), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h]
            at += h
        n_tokens = max(1, sum(new) + case["pad"])
        s.update(ctx_len=_ints(ctx), new_len=_ints(new), free_pages=order[at:].contiguous(),
                 n_free=_ints([n_pages - at]), block_table=table, kv_len=_ints([0] * len(kv)),
                 q_start=_ints([0] * (len(kv) + 1)), slots=_ints([0] * n_tokens), positions=_ints([0] * n_tokens),
                 n_free_out=_ints([0]), cache=_cache(case, n_pages, width, 1))
    elif case["op"] == "write":
        n, hq, hkv, live = case["tokens"] + case["pad"], case["hq"], case["hkv"], case["tokens"]
        n_pages = _up(live, page) + SPARE
        qkv = torch.randn((n, (hq + 2 * hkv) * D), generator=gen, device="cuda", dtype=torch.bfloat16)
        slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:n].to(torch.int32)
        positions = torch.randint(0, 1 << 20, (n,), generator=gen, device="cuda", dtype=torch.int32)
        slots[live:] = -1
        positions[live:] = -1
        weights = [(1 + 0.2 * torch.randn((D,), generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2)]
        freq = _inv_freq(case["rotary"]) if case["rotary"] else []
        s.update(qkv=qkv, slots=slots, positions=positions, q_weight=weights[0] if case["norm"] else None,
                 k_weight=weights[1] if case["norm"] else None, k_pages=_pool(n_pages, hkv, page, gen),
                 v_pages=_pool(n_pages, hkv, page, gen), q_out=torch.zeros((n, hq, D), device="cuda", dtype=torch.bfloat16),
                 inv_freq=torch.tensor(freq, dtype=torch.float64, device="cuda"),
                 cache=_cache(case, n_pages, 1, hq, rotary_dim=case["rotary"], interleaved=case["interleaved"],
                              inv_freq=freq, eps=EPS))
    elif case["op"] == "attention":
        ctx, new = _lengths(case)
        kv = [c + n for c, n in zip(ctx, new)]
        table, n_pages = _table(kv, page, gen)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        n = starts[-1] + case["pad"]
        q = torch.randn((n, case["hq"], D), generator=gen, device="cuda", dtype=torch.bfloat16) * 1.5
        s.update(q=q, k_pages=_pool(n_pages, case["hkv"], page, gen), v_pages=_pool(n_pages, case["hkv"], page, gen),
                 block_table=table, q_start=_ints(starts), kv_len=_ints(kv), out=torch.zeros_like(q),
                 lse=torch.zeros((n, case["hq"]), device="cuda"), max_q=max(new), max_kv=max(kv),
                 cache=_cache(case, n_pages, table.shape[1], case["hq"]))
    else:
        kv = _kv_lengths(case)
        table, n_pages = _table(kv, page, gen)
        shape = (case["batch"], case["layers"], case["hkv"], case["rows"], D)
        s.update(k_pages=_pool(n_pages, case["hkv"], page, gen, case["layers"]),
                 v_pages=_pool(n_pages, case["hkv"], page, gen, case["layers"]), block_table=table, kv_len=_ints(kv),
                 pos0=min(kv) - min(min(kv), case["rows"]), k_out=torch.zeros(shape, device="cuda", dtype=torch.bfloat16),
                 v_out=torch.zeros(shape, device="cuda", dtype=torch.bfloat16),
                 cache=_cache(case, n_pages, table.shape[1], case["hkv"]))
    return s


# ------------------------------------------------------------- one pass ----

def run(state):
    return {"tables": _tables, "write": _write, "attention": _attention, "gather": _gather}[state["op"]](state)


def _tables(s):
    if own:
        s["cache"].tables(s["ctx_len"], s["new_len"], s["free_pages"], s["n_free"], s["block_table"], s["kv_len"],
                          s["q_start"], s["slots"], s["positions"], s["n_free_out"])
        return {k: s[k] for k in ("block_table", "kv_len", "q_start", "slots", "positions", "n_free_out")}
    page, ctx, new = s["case"]["page"], s["ctx_len"].long(), s["new_len"].long()
    kv = ctx + new
    held = (ctx + page - 1) // page
    need = (kv + page - 1) // page - held
    first = need.cumsum(0) - need
    ends = new.cumsum(0)
    col = torch.arange(s["block_table"].shape[1], device="cuda")[None] - held[:, None]
    take = s["n_free"].long() - 1 - first[:, None] - col
    table = torch.where((col >= 0) & (col < need[:, None]),
                        s["free_pages"][take.clamp(0, s["free_pages"].numel() - 1)], s["block_table"])
    t = torch.arange(s["slots"].numel(), device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    live = b < kv.numel()
    b = b.clamp(max=kv.numel() - 1)
    pos = (kv - ends)[b] + t
    slot = table[b, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    return {"block_table": table, "kv_len": kv.int(), "q_start": torch.cat([ends[:1] * 0, ends]).int(),
            "slots": torch.where(live, slot, -1).int(), "positions": torch.where(live, pos, -1).int(),
            "n_free_out": (s["n_free"] - need.sum()).int()}


def _parts(s):
    hq, hkv, n = s["case"]["hq"], s["case"]["hkv"], s["qkv"].shape[0]
    q, k, v = s["qkv"].split([hq * D, hkv * D, hkv * D], 1)
    return q.view(n, hq, D), k.view(n, hkv, D), v.view(n, hkv, D)


def _turned(x, weight, cos, sin, rotary, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    if not rotary:
        return x
    part, rest = x[..., :rotary], x[..., rotary:]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :rotary // 2], part[..., rotary // 2:])
    pair = [a * cos - b * sin, b * cos + a * sin]
    part = torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1)
    return torch.cat([part, rest], -1)


def _write(s):
    q, k, v = _parts(s)
    if own:
        s["cache"].write(q, k, v, s["positions"], s["slots"], s["k_pages"], s["v_pages"], s["q_out"],
                         q_weight=s["q_weight"], k_weight=s["k_weight"])
        return {k: s[k] for k in ("q_out", "k_pages", "v_pages")}
    c, live = s["case"], s["case"]["tokens"]
    angle = s["positions"][:live].double()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    slots = s["slots"][:live].long()
    at, off = slots // c["page"], slots % c["page"]
    s["q_out"][:live] = _turned(q[:live], s["q_weight"], cos, sin, c["rotary"], c["interleaved"]).bfloat16()
    s["k_pages"][at, :, off] = _turned(k[:live], s["k_weight"], cos, sin, c["rotary"], c["interleaved"]).bfloat16()
    s["v_pages"][at, :, off] = v[:live]
    return {k: s[k] for k in ("q_out", "k_pages", "v_pages")}


def _attention(s):
    if own:
        s["cache"].attention(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["q_start"], s["kv_len"],
                             out=s["out"], lse=s["lse"])
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
    for h in range(hkv):  # one kv head's score matrix at a time is what the memory holds
        k, v = s["k_pages"][pages, h, off].float(), s["v_pages"][pages, h, off].float()
        v = torch.where(held, v, 0.0)
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


def _gather(s):
    if own:
        s["cache"].gather(s["k_pages"], s["v_pages"], s["block_table"], s["kv_len"], s["pos0"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    page = s["case"]["page"]
    j = s["pos0"] + torch.arange(s["case"]["rows"], device="cuda")
    pages, off = s["block_table"][:, (j // page).clamp(max=s["block_table"].shape[1] - 1)].long().clamp(min=0), j % page
    held = (j < s["kv_len"][:, None])[..., None, None, None]
    for pool, to in ((s["k_pages"], s["k_out"]), (s["v_pages"], s["v_out"])):
        x = pool.permute(1, 3, 0, 2, 4)[pages, off]               # [request, position, layer, kv head, element]
        to.copy_(torch.where(held, x, 0.0).permute(0, 2, 3, 1, 4))
    return {"k": s["k_out"], "v": s["v_out"]}


# ------------------------------------------------------------- what it takes ----

def work(case):
    if case["op"] == "tables":
        ctx, new = _lengths(case)
        fresh = sum(_up(c + n, case["page"]) - _up(c, case["page"]) for c, n in zip(ctx, new))
        n = max(1, sum(new) + case["pad"])
        return {"bytes": 16 * len(ctx) + 8 * fresh + 8 * n + 12, "flops": 4 * n + 8 * len(ctx)}
    if case["op"] == "write":
        heads, norm = case["hq"] + 2 * case["hkv"], 4 if case["norm"] else 0
        return {"bytes": case["tokens"] * (heads * 2 * D * 2 + 8) + (4 * D if norm else 0) + 4 * case["rotary"],
                "flops": case["tokens"] * (case["hq"] + case["hkv"]) * (norm * D + 3 * case["rotary"] + D)}
    if case["op"] == "attention":
        ctx, new = _lengths(case)
        rows = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
        kv = sum(c + n for c, n in zip(ctx, new))
        pages = sum(_up(c + n, case["page"]) for c, n in zip(ctx, new))
        return {"bytes": sum(new) * case["hq"] * (4 * D + 4) + kv * case["hkv"] * 4 * D + 4 * pages + 8 * len(ctx) + 4,
                "flops": 4 * D * case["hq"] * rows}
    rows = case["batch"] * case["layers"] * case["hkv"] * case["rows"]
    return {"bytes": 8 * D * rows + 4 * case["batch"] * (1 + _up(case["rows"], case["page"])), "flops": rows}


# ------------------------------------------------------ from the definitions ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": lambda _: None, "write": _exact_write, "attention": _exact_attention, "gather": _exact_gather}[
        case["op"]](s)


def _exact_write(s):
    c = s["case"]
    hq, hkv, page, rot = c["hq"], c["hkv"], c["page"], c["rotary"]
    heads = s["qkv"].double().view(-1, hq + 2 * hkv, D)
    q_out, k_pages, v_pages = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
    # the pairs that turn together, and each pair's angle as a complex factor
    first = torch.arange(rot // 2, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else rot // 2)
    factor = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                         torch.outer(s["positions"].double(), s["inv_freq"]))[:, None]

    def turn(x, weight):
        if weight is not None:
            x = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
        z = torch.complex(x[..., first], x[..., second]) * factor
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k, v = turn(heads[:, :hq], s["q_weight"]), turn(heads[:, hq:hq + hkv], s["k_weight"]), heads[:, hq + hkv:]
    live = (s["positions"] >= 0).nonzero().flatten()
    rows = s["slots"][live].long()
    q_out[live] = q[live]
    for pool, x in ((k_pages, k), (v_pages, v)):
        flat = pool.transpose(1, 2).reshape(-1, hkv, D)
        flat[rows] = x[live]
        pool.copy_(flat.view(-1, page, hkv, D).transpose(1, 2))
    return {"q_out": q_out, "k_pages": k_pages, "v_pages": v_pages}


def _exact_attention(s):
    c = s["case"]
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    ctx, new = _lengths(c)
    out, lse = s["out"].double(), s["lse"].double()
    at = 0
    for b in range(c["batch"]):
        n, kv = new[b], ctx[b] + new[b]
        pages = s["block_table"][b, :_up(kv, page)].long()
        for h in range(hq):
            kh = h // (hq // hkv)
            k = s["k_pages"][pages, kh].reshape(-1, D)[:kv].double()
            v = s["v_pages"][pages, kh].reshape(-1, D)[:kv].double()
            x = s["q"][at:at + n, h].double() @ k.T / math.sqrt(D)
            x[:, ctx[b]:] += torch.full((n, n), -math.inf, dtype=torch.float64, device="cuda").triu(1)
            z = torch.logsumexp(x, 1)
            lse[at:at + n, h] = z
            out[at:at + n, h] = x.sub_(z[:, None]).exp_() @ v
        at += n
    return {"out": out, "lse": lse}


def _exact_gather(s):
    c, page = s["case"], s["case"]["page"]
    got = {}
    for name, pool in (("k", s["k_pages"]), ("v", s["v_pages"])):
        x = torch.zeros_like(s["k_out"], dtype=torch.float64)
        for b, kv in enumerate(_kv_lengths(c)):
            pages = s["block_table"][b, :_up(kv, page)].long()
            whole = pool[:, pages].transpose(1, 2).reshape(c["layers"], c["hkv"], -1, D)[:, :, s["pos0"]:kv]
            n = min(c["rows"], whole.shape[2])
            x[b, :, :, :n] = whole[:, :, :n].double()
        got[name] = x
    return got
