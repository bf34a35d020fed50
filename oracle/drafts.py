"""Definitions of the operators that take prompts in and verify trees of drafted
tokens, written out in Python integers and float64 (test infrastructure only)."""
from __future__ import annotations

import math

import numpy as np

PAGE = 16


def _pages(n):
    return (n + PAGE - 1) // PAGE


def ancestors(parents):
    """Of every node itself and those above it; a parent that is not below its node counts as none."""
    above = []
    for i, p in enumerate(map(int, parents)):
        above.append([i] + (above[p] if 0 <= p < i else []))
    return above


def chunk_attention(q, k_pages, v_pages, table, lens, cu, parents=None, scale=None):
    """float64 [tokens, heads, d] arrays; new token i of a request's n sees its first lens - n + i + 1 tokens, or, with
    parents, the first lens - n, itself and the new ones above it.  Tokens of no request: out 0, lse -inf."""
    t, hq, d = q.shape
    hkv = k_pages.shape[1]
    g = hq // hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse = np.zeros((t, hq, d)), np.full((t, hq), -np.inf)
    for b in range(len(lens)):
        first, n, held = int(cu[b]), int(cu[b + 1]) - int(cu[b]), int(lens[b])
        if n == 0 or held <= 0:
            continue
        pages = np.asarray(table[b], dtype=np.int64)[:_pages(held)]
        keys = k_pages[pages].transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :held]
        values = v_pages[pages].transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :held]
        position = np.arange(held) - (held - n)  # of a key among the new tokens; below 0: before them
        if parents is None:
            sees = position[None, :] <= np.arange(n)[:, None]
        else:
            sees = np.tile(position < 0, (n, 1))
            for i, above in enumerate(ancestors(parents[first:first + n])):
                for a in above:
                    sees[i] |= position == a
        rows = slice(first, first + n)
        s = scale * np.einsum("nhgd,hld->nhgl", q[rows].reshape(n, hkv, g, d), keys)
        s = np.where(sees[:, None, None, :], s, -np.inf).reshape(n, hq, held)
        top = s.max(-1, keepdims=True)
        w = np.exp(s - np.where(np.isinf(top), 0, top))
        total = w.sum(-1)
        o = np.einsum("nhgl,hld->nhgd", w.reshape(n, hkv, g, held), values).reshape(n, hq, d)
        some = total > 0
        out[rows] = np.where(some[..., None], o / np.where(some, total, 1)[..., None], 0)
        with np.errstate(divide="ignore"):
            lse[rows] = np.where(some, top[..., 0] + np.log(total), -np.inf)
    return out, lse


def accept_drafts(drafted, parents, cu, sampled):
    """Returns (path, n_kept, next_tokens, n_back) as lists."""
    path, kept, following, back = [-1] * len(drafted), [], [], []
    for b in range(len(cu) - 1):
        first, n = int(cu[b]), int(cu[b + 1]) - int(cu[b])
        steps, at = [], 0 if n else -1
        while at >= 0:
            steps.append(at)
            drawn = int(sampled[first + at])
            at = next((c for c in range(at + 1, n) if int(parents[first + c]) == at and int(drafted[first + c]) == drawn >= 0), -1)
        path[first:first + len(steps)] = steps
        kept.append(len(steps))
        following.append(int(sampled[first + steps[-1]]) if steps else -1)
        back.append(len(steps) - n)
    return path, kept, following, back


def keep_drafts(path, cu, table, lens, k_pages, v_pages):
    """numpy arrays [layers, pages, kv heads, 16, d]; returns the pools after the moves."""
    k, v = k_pages.copy(), v_pages.copy()
    for b in range(len(lens)):
        first, n = int(cu[b]), int(cu[b + 1]) - int(cu[b])
        base = int(lens[b]) - n
        for i in range(n):
            node = int(path[first + i])
            if node < 0:
                break
            a, z = base + node, base + i
            for new, old in ((k, k_pages), (v, v_pages)):
                new[:, int(table[b][z // PAGE]), :, z % PAGE] = old[:, int(table[b][a // PAGE]), :, a % PAGE]
    return k, v


def token_logprobs(row, given=(), temperature=1.0, top=0):
    """One row of logits: (log probabilities of the given tokens, entropy, [(token, log probability)] of the top ones)."""
    row = [float(x) for x in row]
    if any(math.isnan(x) for x in row) or max(row) == -math.inf:
        return [math.nan] * len(given), math.nan, [(-1, math.nan)] * top
    most = max(row)
    order = sorted(range(len(row)), key=lambda i: -row[i])  # stable: ties by index
    if temperature > 0:
        y = [0.0 if x == most else (x - most) / temperature if x > -math.inf else -math.inf for x in row]
        if most == math.inf:
            y = [0.0 if x == most else -math.inf for x in row]
    else:
        y = [0.0 if i == order[0] else -math.inf for i in range(len(row))]
    log_s = math.log(math.fsum(math.exp(x) for x in y))
    entropy = -math.fsum(math.exp(x - log_s) * (x - log_s) for x in y if x > -math.inf)
    best = [(i, y[i] - log_s) for i in order[:top] if row[i] > -math.inf]
    best += [(-1, -math.inf)] * (top - len(best))
    return [y[i] - log_s if 0 <= i < len(row) else math.nan for i in map(int, given)], entropy, best
