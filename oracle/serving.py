"""Plain 64-bit forms of the serving operators: paged-cache append, attention of one new token over a
paged cache, causal window attention of packed prompts, and the MoE layer for a few tokens.

Each attention form also returns how far a kernel may be off that rounds its weights to the
activations' type (half a step u) and sums in fp32, element by element:

  a score sums d exact products of fp32 precision: off by at most e = d 2^-23 max sum |q k| scale (each
  addition rounds or truncates by at most 2^-23 of a partial sum), and 2^-21 |s| for its scaling;
  a weight is then off by 2 e relative (the score's and the normaliser's), its exponential by 2^-20, its
  rounding by u:  |out - exact| <= (u + 2 e + 2^-20) sum p |v| + u |out|;
  |lse - exact| <= e + 2^-20 (1 + |lse|).

Weights held in fp16 (fp16 activations, or an e4m3 cache) have a step of 2^-24 below 2^-14, whatever their
size.  The kernels hold them times 2^7, so it is 2^-32 more for each key's weight; and 2^-25 for an fp16 output.
"""
from __future__ import annotations

import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "f32": 2.0 ** -24}


def visible(pos: int, count: int, window: int, sinks: int) -> np.ndarray:
    """The keys (indices below count) that a query standing at key `pos` sees."""
    j = np.arange(count)
    seen = j <= pos
    if window:
        seen &= (j > pos - window) | (j < sinks)
    return j[seen]


def attend(q, k, v, scale, u, fp16_weights=False):
    """One query row q [d] over the rows k, v [m, d] (float64): out, lse and their tolerances."""
    d = q.shape[0]
    if k.shape[0] == 0:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        s = k @ q * scale
        top = s.max()
        w = np.exp(s - top)
        total = w.sum()
        p = w / total
        out = p @ v
        lse = top + np.log(total)
        finite = np.isfinite(s)
        sums = (np.abs(k) @ np.abs(q))[finite]
        e = (d * 2.0 ** -23 * sums.max() + 2.0 ** -21 * np.abs(s[finite] / scale).max()) * scale if sums.size else 0.0
        tol = (u + 2 * e + 2.0 ** -20) * (p @ np.abs(v)) + u * np.abs(out)
        if fp16_weights:
            tol = tol + 2.0 ** -32 * np.abs(v).sum(0) / total + 2.0 ** -25
    return out, lse, tol, e + 2.0 ** -20 * (1 + abs(lse))


def paged_attention(q, k_cache, v_cache, table, lengths, scale, window=0, sinks=0, k_scale=None, v_scale=None, u=2.0 ** -8,
                    fp16_weights=False, bad_pages=()):
    """q [B, Hq, d], caches [pages, page, Hk, d] (float64 values of the stored rows), pages in bad_pages absent."""
    B, Hq, d = q.shape
    pages, page, Hk, _ = k_cache.shape
    out, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    tol, ltol = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        n = int(lengths[b])
        rows = visible(n - 1, n, window, sinks)
        rows = np.array([r for r in rows if table[b][r // page] not in bad_pages], dtype=np.int64)
        at = np.asarray(table[b])[rows // page] if rows.size else rows
        for h in range(Hq):
            hk = h // (Hq // Hk)
            k, v = k_cache[at, rows % page, hk], v_cache[at, rows % page, hk]
            if k_scale is not None:
                k = k * k_scale[hk]
            if v_scale is not None:
                v = v * v_scale[hk]
            out[b, h], lse[b, h], tol[b, h], ltol[b, h] = attend(q[b, h], k, v, scale, u, fp16_weights)
    return out, lse, tol, ltol


def window_attention(q, k, v, cu_q, cu_k, scale, window=0, sinks=0, u=2.0 ** -8, fp16_weights=False):
    """Packed sequences: q [nq, Hq, d], k and v [nk, Hk, d]."""
    nq, Hq, d = q.shape
    g = Hq // k.shape[1]
    out, lse = np.zeros((nq, Hq, d)), np.full((nq, Hq), -np.inf)
    tol, ltol = np.zeros((nq, Hq, d)), np.zeros((nq, Hq))
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(n):
            seen = visible(m - n + i, m, window, sinks) + cu_k[b]
            t = cu_q[b] + i
            for h in range(Hq):
                out[t, h], lse[t, h], tol[t, h], ltol[t, h] = attend(q[t, h], k[seen, h // g], v[seen, h // g], scale,
                                                                       u, fp16_weights)
    return out, lse, tol, ltol


def moe_tokens(x, logits, w_gate, w_up, w_down, topk, renorm=False):
    """The layer, and how far a kernel may be off that sums in fp32 (a sum of n terms is off by at most
    n 2^-23 of the sum of their absolute values, whatever its order), carried through SiLU, whose
    slope is at most 1.1, and the two products; h itself is kept to 2^-21."""
    T, H = x.shape
    F = w_gate.shape[2]
    step = 2.0 ** -23
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    experts, gates = np.zeros((T, topk), dtype=np.int32), np.zeros((T, topk))
    for t in range(T):
        row = np.asarray(logits[t], dtype=np.float64)
        w = np.exp(row - row.max())
        w /= w.sum()
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:topk]
        total = sum(w[e] for e in best) if renorm else 1.0
        for j, e in enumerate(best):
            a, b = x[t] @ w_gate[e], x[t] @ w_up[e]
            ea, eb = H * step * (np.abs(x[t]) @ np.abs(w_gate[e])), H * step * (np.abs(x[t]) @ np.abs(w_up[e]))
            silu = a / (1 + np.exp(-a))
            h = silu * b
            eh = 1.1 * ea * (np.abs(b) + eb) + np.abs(silu) * eb + 2.0 ** -21 * np.abs(h)
            y = h @ w_down[e]
            ey = eh @ np.abs(w_down[e]) + F * step * (np.abs(h) @ np.abs(w_down[e]))
            g = w[e] / total
            experts[t, j], gates[t, j] = e, g
            out[t] += g * y
            tol[t] += g * ey + 2.0 ** -19 * g * np.abs(y)
    return out, experts, gates, tol
