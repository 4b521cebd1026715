"""fp64 statement of the latent-attention calls (numpy, one row at a time).

``absorbed`` and ``expanded`` also return, for every output row, what error
bounds need: sum_j p_j |v_j| per value (an output that rounds every p_j and the
result to bf16 is off by at most a known part of it) and the largest
scale * sum_d |q_d k_jd| of the row (bounds the rounding of fp32 scores).
"""
from __future__ import annotations

import numpy as np

LAT, PE, NOPE = 512, 64, 128


def plan(cached, new, table, free, page, capacity):
    """Lists in, dict of lists out; ``table`` (a list of lists) is not changed."""
    rows = [list(r) for r in table]
    slots, cu, taken = [], [0], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        for at in range(-(-c // page), -(-(c + n) // page)):
            rows[b][at] = free[taken]
            taken += 1
        slots += [rows[b][pos // page] * page + pos % page for pos in range(c, c + n)]
        cu.append(cu[-1] + n)
    return dict(table=rows, seq_lens=[c + n for c, n in zip(cached, new)], cu_seqlens=cu,
                slot_map=slots + [-1] * (capacity - len(slots)), pages_taken=[taken])


def normalised(c, weight, eps):
    c = np.asarray(c, np.float64)
    return c / np.sqrt((c ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def _attend(q, keys, values, scale):
    """Rows q [r, d] against keys [n, d], values [n, w]: out, lse, spread, reach."""
    r, w = q.shape[0], values.shape[1]
    if keys.shape[0] == 0:
        return np.zeros((r, w)), np.full(r, -np.inf), np.zeros((r, w)), np.zeros(r)
    s = scale * (q @ keys.T)
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    z = e.sum(1, keepdims=True)
    p = e / z
    return p @ values, (top + np.log(z))[:, 0], p @ np.abs(values), (scale * (np.abs(q) @ np.abs(keys).T)).max(1)


def absorbed(q, cache, table, lens, scale):
    """q [B, R, H, 576], cache [pages, page, 576], table [B, max], lens [B]."""
    B, R, H, _ = q.shape
    page = cache.shape[1]
    out, spread = np.zeros((B, R, H, LAT)), np.zeros((B, R, H, LAT))
    lse, reach = np.zeros((B, R, H)), np.zeros((B, R, H))
    for b in range(B):
        n = int(lens[b])
        rows = np.array([cache[table[b][j // page], j % page] for j in range(n)]).reshape(n, LAT + PE)
        for i in range(R):
            seen = rows[:max(0, n - (R - 1 - i))]
            out[b, i], lse[b, i], spread[b, i], reach[b, i] = _attend(q[b, i], seen, seen[:, :LAT], scale)
    return out, lse, spread, reach


def expanded(q, k, k_pe, v, scale, causal, cu_q=None, cu_k=None):
    """q [B, Tq, H, 192], k and v [B, Tk, H, 128], k_pe [B, Tk, 64]."""
    B, Tq, H, _ = q.shape
    out, spread = np.zeros((B, Tq, H, v.shape[3])), np.zeros((B, Tq, H, v.shape[3]))
    lse, reach = np.zeros((B, Tq, H)), np.zeros((B, Tq, H))
    if cu_q is None:
        seqs = [(b, 0, Tq, 0, k.shape[1]) for b in range(B)]
    else:
        seqs = [(0, cu_q[n], cu_q[n + 1], cu_k[n], cu_k[n + 1]) for n in range(len(cu_q) - 1)]
    for b, q0, q1, k0, k1 in seqs:
        for h in range(H):
            keys = np.concatenate([k[b, k0:k1, h], k_pe[b, k0:k1]], -1)
            for i in range(q0, q1):
                seen = min(k1 - k0, i - q0 + 1 + (k1 - k0) - (q1 - q0)) if causal else k1 - k0
                seen = max(0, seen)
                o, z, sp, re = _attend(q[b, i:i + 1, h], keys[:seen], v[b, k0:k0 + seen, h], scale)
                out[b, i, h], lse[b, i, h], spread[b, i, h], reach[b, i, h] = o[0], z[0], sp[0], re[0]
    return out, lse, spread, reach


# ---- pages that several requests hold: lists in, lists out, nothing changed in place ----

def fork(parents, children, take, cached, table, free, shares, page):
    """Also returns the copies as (page, from page, rows)."""
    rows, counts, lens, copies = [list(r) for r in table], list(shares), list(cached), []
    for f, (parent, child) in enumerate(zip(parents, children)):
        tokens = cached[parent] if take is None else take[f]
        for at in range(tokens // page):
            rows[child][at] = table[parent][at]
            counts[table[parent][at]] += 1
        if tokens % page:
            rows[child][tokens // page] = free[len(copies)]
            copies.append((free[len(copies)], table[parent][tokens // page], tokens % page))
        lens[child] = tokens
    return dict(table=rows, shares=counts, seq_lens=lens, pages_taken=[len(copies)], copies=copies)


def release(which, keep, cached, table, shares, page):
    counts, lens = list(shares), list(cached)
    for f, b in enumerate(which):
        kept = 0 if keep is None else keep[f]
        for at in range(-(-kept // page), -(-cached[b] // page)):
            counts[table[b][at]] -= 1
        lens[b] = kept
    free = [p for p, c in enumerate(counts) if c < 0]
    return dict(shares=[max(0, c) for c in counts], seq_lens=lens, pages=free + [-1] * (len(counts) - len(free)),
                count=[len(free)])


def compact(cached, table, shares, page):
    """Also returns the moves as (to page, from page)."""
    held = sorted({table[b][at] for b, n in enumerate(cached) for at in range(-(-n // page))})
    used = len(held)
    places = [p for p in range(used) if p not in set(held)]
    moves = list(zip(places, [p for p in held if p >= used]))
    new = {p: p for p in held}
    new.update({was: to for to, was in moves})
    counts = [0] * len(shares)
    for was, to in new.items():
        counts[to] = shares[was]
    rows = [[new[p] if at < -(-cached[b] // page) else p for at, p in enumerate(r)] for b, r in enumerate(table)]
    return dict(table=rows, shares=counts, page_map=[new.get(p, -1) for p in range(len(shares))], pages_used=[used],
                moves=moves)
