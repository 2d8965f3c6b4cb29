"""fp64 oracle of the operators around a paged K/V cache (NumPy, test
infrastructure only): norms with rotation, packed causal attention, attention
of drafted tokens, collected weights and eviction, each straight from its
definition and one sequence and head at a time.  Shares no code with the CUDA
path."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def norm_rope(x, positions, inv_freq, weight=None, eps=0.0, interleaved=False):
    """x [n][H][d] float64 -> normalised (weight given) and rotated rows."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = len(inv_freq)
    out = y.copy()
    for r, t in enumerate(positions):
        for f in range(half):
            u = float(int(t)) * float(inv_freq[f])
            c, s = np.cos(u), np.sin(u)
            a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
            out[r, :, a] = y[r, :, a] * c - y[r, :, b] * s
            out[r, :, b] = y[r, :, b] * c + y[r, :, a] * s
    return out


def masked_attn(q, k, v, seen):
    """One head: q [n][d], k, v [m][d], seen bool [n][m] -> o [n][d], lse [n];
    a query that sees nothing gives zeros and -inf."""
    o, lse = np.zeros((q.shape[0], v.shape[1])), np.full(q.shape[0], -np.inf)
    for i in range(q.shape[0]):
        js = np.nonzero(seen[i])[0]
        if js.size == 0:
            continue
        s = k[js] @ q[i] / np.sqrt(q.shape[1])
        m = s.max()
        e = np.exp(s - m)
        o[i], lse[i] = e @ v[js] / e.sum(), m + np.log(e.sum())
    return o, lse


def varlen_attn(q, k, v, cu_q, cu_k):
    """q [total_q][Hq][d], k, v [total_k][Hkv][d]; rows outside the sequences are NaN in the result."""
    Hq, G = q.shape[1], q.shape[1] // k.shape[1]
    o, lse = np.full(q.shape, np.nan), np.full((Hq, q.shape[0]), np.nan)
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        seen = np.arange(nk)[None, :] <= np.arange(nq)[:, None] + (nk - nq)
        for h in range(Hq):
            qs, ks = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
            o[qs, h], lse[h, qs] = masked_attn(q[qs, h], k[ks, h // G], v[ks, h // G], seen)
    return o, lse


def draft_seen(ctx, masks, t):
    """Which of the ctx + t keys each of t drafted tokens sees; masks None: a chain."""
    seen = np.zeros((t, ctx + t), dtype=bool)
    seen[:, :ctx] = True
    for i in range(t):
        for j in range(t):
            seen[i, ctx + j] = j <= i if masks is None else bool(int(masks[i]) >> j & 1)
    return seen


def rows_of(table, page, n):
    """Pool tokens of positions 0 .. n - 1 of one sequence."""
    return np.array([int(table[p // page]) * page + p % page for p in range(n)], dtype=np.int64)


def tree_attn(q, k, v, table, page, ctx_len, cu, masks):
    """q [n][Hq][d]; k, v pools [tokens][Hkv][d]; NaN rows outside the sequences."""
    Hq, G = q.shape[1], q.shape[1] // k.shape[1]
    o, lse = np.full(q.shape, np.nan), np.full((Hq, q.shape[0]), np.nan)
    for b, ctx in enumerate(ctx_len):
        rs = slice(cu[b], cu[b + 1])
        t = cu[b + 1] - cu[b]
        seen = draft_seen(ctx, None if masks is None else masks[rs], t)
        at = rows_of(table[b], page, ctx + t)
        for h in range(Hq):
            o[rs, h], lse[h, rs] = masked_attn(q[rs, h], k[at, h // G], v[at, h // G], seen)
    return o, lse


def cache_weights(q, k, table, page, ctx_len, cu, masks, lse, counted, acc):
    """acc [B][Hkv][stride] plus the collected weights."""
    out = np.array(acc, dtype=np.float64)
    Hq, G, d = q.shape[1], q.shape[1] // k.shape[1], q.shape[2]
    for b, ctx in enumerate(ctx_len):
        t = cu[b + 1] - cu[b]
        seen = draft_seen(ctx, None if masks is None else masks[cu[b]:cu[b + 1]], t)
        at = rows_of(table[b], page, ctx + t)
        for i in range(t):
            r = cu[b] + i
            if counted is not None and not counted[r]:
                continue
            for h in range(Hq):
                if lse[h, r] == -np.inf:
                    continue
                p = np.exp(k[at, h // G] @ q[r, h] / np.sqrt(d) - lse[h, r])
                out[b, h // G, :ctx + t] += np.where(seen[i], p, 0.0)
    return out


def kept_positions(acc_row, n, keep, recent):
    """Positions that stay, ascending, by a stable ranking."""
    if n <= keep:
        return list(range(n))
    ranked = sorted(range(n - recent), key=lambda j: (-float(acc_row[j]), j))
    return sorted(ranked[:keep - recent]) + list(range(n - recent, n))
