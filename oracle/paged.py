"""Float64 statement of the paged-cache operators (numpy, loops over requests and heads).

Written from the operators' formulas alone; the tests compare the CUDA kernels
with it.  Pools are [n_pages][n_kv_heads][page][128]; a request's position p is
row p % page of page table[b][p // page]."""
from __future__ import annotations

import numpy as np

D = 128


def page_tables(ctx, new, free, n_free, table, page, n_tokens):
    """One step's pages, slots and positions from the requests' lengths; the table is a copy."""
    table = np.array(table, np.int64)
    slots, positions, q_start = np.full(n_tokens, -1, np.int64), np.full(n_tokens, -1, np.int64), [0]
    left, t = int(n_free), 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        for p in range(c, c + n):
            j = p // page
            if p % page == 0:       # the position opens a page
                left -= 1
                table[b, j] = free[left]
            slots[t], positions[t] = table[b, j] * page + p % page, p
            t += 1
        q_start.append(t)
    return {"block_table": table, "kv_len": np.add(ctx, new), "q_start": np.array(q_start), "slots": slots,
            "positions": positions, "n_free_out": np.array([left])}


def norm_rotate(x, weight, eps, positions, inv_freq, interleaved=False, scale=1.0):
    """x [n][heads][128] float64: x / rms(x) * weight (weight None: x), then the rotation of the first
    2 * len(inv_freq) elements by positions * inv_freq.  Also returns the normed x."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * weight
    normed = x.copy()
    h = len(inv_freq)
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        # whole turns dropped exactly: the angle of position p is p * f modulo one turn, in rationals
        angle = np.array([_angle(int(p), float(inv_freq[i])) for p in positions])[:, None]
        c, s = scale * np.cos(angle), scale * np.sin(angle)
        x[..., a], x[..., b] = normed[..., a] * c - normed[..., b] * s, normed[..., b] * c + normed[..., a] * s
    return x, normed


def _angle(p, f):
    """p * f (radians) as a small angle: the product in exact rationals, whole turns of a 200-bit pi taken off."""
    from fractions import Fraction

    two_pi = Fraction(2 * 3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)
    a = Fraction(f) * p
    return float(a - two_pi * round(a / two_pi))


def rows_of(pool, table_row, kh, n):
    """The n cached rows of one request and kv head, in position order."""
    page = pool.shape[2]
    return np.concatenate([pool[int(table_row[j]), kh] for j in range(-(-n // page))] or [np.zeros((0, D))])[:n]


def attention(q, k_pages, v_pages, table, q_start, kv_len):
    """out, lse of every live token, and spread = sum of weight * |v| (what a relative error of the
    weights is relative to); rows behind the last request are NaN."""
    n, hq, hkv = q.shape[0], q.shape[1], k_pages.shape[1]
    out, spread, lse = np.full((n, hq, D), np.nan), np.full((n, hq, D), np.nan), np.full((n, hq), np.nan)
    for b, kv in enumerate(kv_len):
        s, e = int(q_start[b]), int(q_start[b + 1])
        seen = np.arange(int(kv))[None] <= (int(kv) - (e - s) + np.arange(e - s))[:, None]
        for h in range(hq):
            kh = h // (hq // hkv)
            k, v = rows_of(k_pages, table[b], kh, int(kv)), rows_of(v_pages, table[b], kh, int(kv))
            with np.errstate(invalid="ignore"):   # infinities and NaN at unseen positions
                x = q[s:e, h] @ k.T / np.sqrt(D)
            x = np.where(seen, x, -np.inf)
            top = np.max(x, axis=1, initial=-np.inf, keepdims=True)
            w = np.exp(x - np.where(np.isfinite(top), top, 0.0))
            z = w.sum(1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[s:e, h] = (np.where(np.isfinite(top), top, 0.0) + np.log(z))[:, 0]
            w = w / np.where(z > 0, z, 1.0)
            # a position that no row sees does not enter; one that some rows see is added row by row
            fine = np.isfinite(v).all(1)
            out[s:e, h] = w[:, fine] @ v[fine]
            spread[s:e, h] = w[:, fine] @ np.abs(v[fine])
            for j in np.nonzero(~fine)[0]:
                out[s:e, h][seen[:, j]] += w[seen[:, j], j][:, None] * v[j]
    return out, lse, spread


def gather(pools, table, kv_len, pos0, n):
    """[batch][layers][n_kv_heads][n][128] from pools [layers][n_pages][n_kv_heads][page][128]."""
    layers, hkv = pools.shape[0], pools.shape[2]
    out = np.zeros((len(kv_len), layers, hkv, n, D), pools.dtype)
    for b, kv in enumerate(kv_len):
        for layer in range(layers):
            for h in range(hkv):
                r = rows_of(pools[layer], table[b], h, int(kv))[pos0:pos0 + n]
                out[b, layer, h, :len(r)] = r
    return out


# ------------------------------------------------------------------ in 8 bits ----
#
# A pool in 8 bits is (values [n_pages][n_kv_heads][page][128], exponents [n_pages][n_kv_heads][page // 16]): a row is
# its values times 2 ** exponent of its group of sixteen positions.

GROUP = 16
LOWEST = -64   # the smallest exponent


def e4m3(x):
    """The nearest number of four significant bits at 2^-6 or above, multiple of 2^-9 below that (ties to even)."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(x), np.rint(x / step) * step, np.nan)


def exponent(top):
    """The smallest exponent e >= LOWEST with top <= 448 * 2^e."""
    e = LOWEST
    while top > np.ldexp(448.0, e):
        e += 1
    return e


def append8(values, exps, x, slots):
    """The pool (values, exps) after the rows x [token][n_kv_heads][128] came to their slots (-1: nowhere)."""
    values, exps = np.array(values, np.float64), np.array(exps, np.int64)
    page = values.shape[2]
    groups = {}
    for t, s in enumerate(slots):
        if s >= 0:
            groups.setdefault(int(s) // GROUP, []).append((int(s) % GROUP, t))
    for g, rows in groups.items():
        at, sub = divmod(g, page // GROUP)
        begin = min(o for o, _ in rows)
        here = slice(sub * GROUP, (sub + 1) * GROUP)
        for h in range(values.shape[1]):
            new = np.array([x[t, h] for _, t in rows])
            e = exponent(np.abs(new[np.isfinite(new)]).max(initial=0.0))
            if begin > 0:
                e = max(e, int(exps[at, h, sub]))
                held = values[at, h, here][:begin]
                values[at, h, here][:begin] = e4m3(np.ldexp(held, int(exps[at, h, sub]) - e))
            exps[at, h, sub] = e
            for (o, _), row in zip(rows, new):
                values[at, h, sub * GROUP + o] = e4m3(np.ldexp(row, -e))
    return values, exps


def widened(values, exps):
    """The rows that a pool in 8 bits stands for."""
    return np.ldexp(np.asarray(values, np.float64), np.repeat(np.asarray(exps, np.int64), GROUP, axis=-1)[..., None])
