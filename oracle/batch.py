"""Definitions of the operators whose lengths live on the GPU, written out in
Python integers and float64 (test infrastructure only)."""
from __future__ import annotations

import math

import numpy as np

PAGE = 16


def _pages(n):
    return (n + PAGE - 1) // PAGE


def extend_tables(lens, n_new, table, free, n_free, max_new, base=0):
    """Returns (slots, positions, cu_new, lens, table, free, n_free) after the step, or None where it cannot be done
    (pages, table rows or outputs do not suffice, a length is out of range)."""
    lens, table, free = [int(x) for x in lens], [list(map(int, r)) for r in table], [int(x) for x in free]
    width, n_free = len(table[0]) if table else 0, int(n_free)
    if not 0 <= n_free <= len(free):
        return None
    taken, given, after = [], [], []
    for b, (held, n) in enumerate(zip(lens, map(int, n_new))):
        now = max(held + n, 0)
        if held < 0 or max(held, now) > width * PAGE:
            return None
        taken += [(b, j) for j in range(_pages(held), _pages(now))]
        given += [(b, j) for j in range(_pages(now), _pages(held))]
        after.append(now)
    if len(taken) > n_free or n_free - len(taken) + len(given) > len(free):
        return None
    if sum(max(int(n), 0) for n in n_new) > max_new:
        return None
    top = n_free
    for b, j in taken:
        top -= 1
        table[b][j] = free[top]
    for b, j in reversed(given):
        free[top] = table[b][j]
        top += 1
    slots, positions, cu = [], [], [0]
    for b, (held, now) in enumerate(zip(lens, after)):
        for pos in range(held, now):
            slots.append(table[b][pos // PAGE] * PAGE + pos % PAGE)
            positions.append(base + pos)
        cu.append(len(slots))
    pad = [-1] * (max_new - len(slots))
    return slots + pad, positions + pad, cu, after, table, free, top


def append_slots(k_new, v_new, slots, k_pages, v_pages):
    """numpy arrays; returns the pools after the writes."""
    k, v = k_pages.copy(), v_pages.copy()
    for t, s in enumerate(map(int, slots)):
        if 0 <= s < k.shape[0] * PAGE:
            k[s // PAGE, :, s % PAGE] = k_new[t]
            v[s // PAGE, :, s % PAGE] = v_new[t]
    return k, v


def prefix_attention(q, k_pages, v_pages, table, lens, cu, prefix_pages, prefix_len, scale=None):
    """float64 [tokens, heads, d] arrays; token t of request b (of n, the j-th) sees the prefix and the request's first
    lens[b] - n + j + 1 tokens.  Tokens of no request: out 0, lse -inf."""
    t, hq, d = q.shape
    g = hq // k_pages.shape[1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse = np.zeros((t, hq, d)), np.full((t, hq), -np.inf)

    def rows(pool, pages, h, n):
        pages = np.asarray(pages, dtype=np.int64)[:_pages(n)]
        return pool[pages, h].reshape(-1, d)[:n]

    for b in range(len(lens)):
        n = int(cu[b + 1]) - int(cu[b])
        for j in range(n):
            row, end = int(cu[b]) + j, max(int(lens[b]) - n + j + 1, 0)
            for h in range(hq):
                keys = np.concatenate([rows(k_pages, prefix_pages, h // g, prefix_len), rows(k_pages, table[b], h // g, end)])
                values = np.concatenate([rows(v_pages, prefix_pages, h // g, prefix_len), rows(v_pages, table[b], h // g, end)])
                if not len(keys):
                    continue
                s = scale * (keys @ q[row, h])
                w = np.exp(s - s.max())
                out[row, h] = w @ values / w.sum()
                lse[row, h] = s.max() + math.log(w.sum())
    return out, lse


def sample(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row of logits and its random numbers: [(token, ln of its probability among the kept)] per number."""
    row = [float(x) for x in row]
    if any(math.isnan(x) for x in row) or max(row) == -math.inf:
        return [(-1, math.nan)] * len(u)
    top = max(row)
    order = sorted(range(len(row)), key=lambda i: -row[i])  # stable: ties by index
    if not temperature > 0:
        return [(order[0], 0.0)] * len(u)
    weight = [1.0 if x == top else math.exp((x - top) / temperature) if x > -math.inf else 0.0 for x in row]
    kept = order[:top_k] if top_k > 0 else order
    if top_p < 1:
        total, before, size = math.fsum(weight[i] for i in kept), 0.0, 0
        for i in kept:
            if size and not before < top_p * total:
                break
            before += weight[i]
            size += 1
        kept = kept[:size]
    kept = sorted({order[0], *(i for i in kept if weight[i] >= min_p)})
    total, got = math.fsum(weight[i] for i in kept), []
    for x in u:
        c = 0.0
        last = None
        for i in kept:
            c += weight[i]
            if weight[i] > 0:
                last = i
                if c > float(x) * total:
                    break
        got.append((last, math.log(weight[last] / total)))
    return got
