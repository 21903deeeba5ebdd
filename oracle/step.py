"""Plain 64-bit forms of what a serving step needs around its attention: the plan of its tokens in a paged cache, norms
and rotation of queries and keys, rows held in 4 bits, and log probabilities of chosen tokens.

The forms that compute numbers also return how far a kernel may be off that works in fp32, element by element.
"""
from __future__ import annotations

import numpy as np

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------------------------------------ 4 bits
def e4m3(x):
    """The byte of the nearest e4m3 value of x >= 0 (fp32 array; ties to even, saturating at 448, NaN 0x7f)."""
    out = np.zeros(x.shape, np.uint8)
    for i, v in np.ndenumerate(np.asarray(x, np.float64)):
        if np.isnan(v):
            out[i] = 0x7F
        elif v >= 448.0:
            out[i] = 0x7E
        elif v < 2.0 ** -6:
            out[i] = int(np.round(v * 512))                     # steps of 2^-9 (numpy rounds ties to even)
        else:
            e = int(np.floor(np.log2(v)))
            out[i] = min(0x7E, ((e + 7) << 3) + int(np.round((v / 2.0 ** e - 1.0) * 8)))
    return out


def e4m3_value(b):
    b = np.asarray(b, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


def to_4_bits(x, scale):
    """Rows x [..., kv_heads, d] (values of a 16-bit type) as codes [..., kv_heads, d / 2] and block scales (bytes)
    [..., kv_heads, d / 16], each quotient and product in fp32 as the layout defines it."""
    with np.errstate(all="ignore"):
        x = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 16)
        s = np.asarray(scale, np.float32)[:, None]
        b = e4m3(np.abs(x).max(-1) / (np.float32(6) * s))
        t = (e4m3_value(b).astype(np.float32) * s)[..., None]
        q = np.where(t == 0, np.float32(0), x / t)
        a = np.abs(q)
        c = ((a > 0.25).astype(np.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).astype(np.uint8)
        c = (c + 8 * np.signbit(q)).astype(np.uint8).reshape(*c.shape[:-2], -1)
    return c[..., ::2] | (c[..., 1::2] << 4), b


def from_4_bits(codes, blocks, scale=None):
    """The values that codes and block scales stand for (with the heads' scales if given)."""
    codes = np.asarray(codes, np.int64)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = CODES[c & 7] * np.where(c & 8, -1.0, 1.0)
    v = v * np.repeat(e4m3_value(blocks), 16, -1)
    return v if scale is None else v * np.asarray(scale, np.float64)[:, None]


# ------------------------------------------------------------------------------------------------ plan
def cache_plan(lengths, counts, table, page, free, taken, tokens, kv_tokens=None):
    """What tl_cache_plan writes, token by token; `ok`: nothing was out of range."""
    table, batch = np.array(table), len(lengths)
    cap, left, ok = table.shape[1] * page, len(free) - taken, True
    if not 0 <= taken <= len(free):
        left, ok = 0, False
    slots, positions, kv = np.full(tokens, -1), np.zeros(tokens, int), []
    cu_q, cu_k, new, used, asked = [0], [0], [], 0, 0
    for b in range(batch):
        n, c = int(lengths[b]), int(counts[b])
        was = n
        if n < 0 or c < 0 or n + c > cap:
            ok, c = False, 0
            n = n if 0 <= n <= cap else 0
        has, needs = -(-n // page), -(-(n + c) // page)
        asked += needs - has
        fits = cu_q[-1] + c <= tokens and (needs == has or asked <= left)
        if c and not fits:
            ok = False
        gets = c if fits else 0
        if gets:
            for i in range(has, needs):
                table[b, i] = free[taken + asked - (needs - has) + i - has]
            if needs > has:
                used = asked
        for i in range(c):
            t = cu_q[-1] + i
            if t < tokens:
                positions[t] = n + i
                if gets:
                    p = int(table[b, (n + i) // page])
                    s = p * page + (n + i) % page
                    slots[t] = s if p >= 0 and s < 2 ** 31 else -1
                    ok &= slots[t] >= 0
        for j in range(n + gets):
            p = int(table[b, j // page])
            kv.append(p * page + j % page if p >= 0 else -1)
        cu_q.append(cu_q[-1] + c)
        cu_k.append(cu_k[-1] + n + gets)
        new.append(was if not gets else n + gets)
    out = dict(table=table, slots=slots, positions=positions, cu_q=np.array(cu_q), cu_k=np.array(cu_k), lengths=np.array(new, int),
               taken=np.array([taken + used]))
    if kv_tokens is not None:
        ok &= len(kv) <= kv_tokens
        out["kv_slots"] = np.array((kv + [-1] * kv_tokens)[:kv_tokens], int)
        ok &= all(s >= 0 for s in kv[:kv_tokens])
    return out, ok


# ------------------------------------------------------------------------------------------------ norms and rotation
def norm_rope(x, weight, positions, inv_freq, eps, interleaved, u):
    """Rows x [tokens, heads, d] (float64), and how far off fp32 work rounded once to half a step u may be: the mean of d
    squares by d / 2 + 4 roundings of 2^-24, its root and three products by 2^-21 together, a turn by
    2^-21 for sine or cosine and 2^-22 for the angle, each of both of a pair's values."""
    n, h, d = x.shape
    y = np.array(x, np.float64)
    rel = 2.0 ** -24
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
        rel = (d / 2 + 4) * 2.0 ** -24 + 2.0 ** -21
    mass = np.abs(y)
    pairs = 0 if inv_freq is None else len(inv_freq)
    if pairs:
        angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
        far = np.abs(angle) * 2.0 ** -53
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        i = np.arange(pairs)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, ya * s + yb * c
        both = np.abs(ya) + np.abs(yb)
        mass[..., a] = mass[..., b] = both
        turn = np.zeros(mass.shape)
        turn[..., a] = turn[..., b] = (2.0 ** -21 + 2.0 ** -22 + far)[:, None] * both
    else:
        turn = 0.0
    return y, u * np.abs(y) + mass * (rel + 2.0 ** -22) * (1 + u) + turn * (1 + u) + 2.0 ** -25


# ------------------------------------------------------------------------------------------------ log probabilities
def token_logprobs(x, targets, top, scale):
    """Rows x [rows, vocab] (float64).  With l = scale log2 e, fp32 leaves z = l (x - m) off by 2^-22 |z| (a
    difference, l and a product), which moves a weight by at most 2^-22 |z| 2^z ln 2 <= 2^-22, a power of two by 2^-22, and a sum of V terms, by V / 256 of them
    in a thread and then in pairs, by (V / 256 + 64) 2^-24 of itself."""
    rows, vocab = x.shape
    got = {w: np.zeros(rows) for w in ("logprob", "entropy", "lse")}
    tol = {w: np.zeros(rows) for w in ("logprob", "entropy", "lse")}
    ids, best, btol = np.zeros((rows, top), np.int64), np.zeros((rows, top)), np.zeros((rows, top))
    for r in range(rows):
        with np.errstate(all="ignore"):
            y = np.asarray(x[r], np.float64) * scale
            order = np.lexsort((np.arange(vocab), np.where(np.isnan(y), np.inf, -y), np.isnan(y)))[:top]
            ids[r] = order
            if np.all(y == -np.inf):
                got["logprob"][r], got["entropy"][r], got["lse"][r], best[r] = -np.inf, 0.0, -np.inf, -np.inf
                continue
            if not np.all(y < np.inf):                           # a NaN or +inf
                for w in got:
                    got[w][r] = np.nan
                best[r] = np.nan
                continue
            m = y.max()
            w = np.exp(y - m)
            total = w.sum()
            p, lse = w / total, m + np.log(total)
            lp = y - lse
            seen = p > 0
            got["lse"][r] = lse
            got["entropy"][r] = -(p[seen] * lp[seen]).sum()
            got["logprob"][r] = lp[targets[r]] if targets is not None else 0.0
            best[r] = lp[order]
            z = 2.0 ** -22 * (p[seen] * np.abs(y[seen] - m)).sum() + 2.0 ** -22
            s = z + 2.0 ** -22 + (vocab / 256 + 64) * 2.0 ** -24
            tol["lse"][r] = s + 2.0 ** -22 * (abs(lse) + 1)
            tol["entropy"][r] = tol["lse"][r] + z + 2 * s * (p[seen] * np.abs(y[seen] - m)).sum() + 2.0 ** -22 * got["entropy"][r]
            tol["logprob"][r] = tol["lse"][r] + z + 2.0 ** -21 * abs(got["logprob"][r]) if np.isfinite(got["logprob"][r]) else 0.0
            btol[r] = np.where(np.isfinite(best[r]), tol["lse"][r] + z + 2.0 ** -21 * np.abs(np.where(np.isfinite(best[r]), best[r], 0)), 0.0)
    return got, tol, ids, best, btol
