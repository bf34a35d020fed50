"""Cases for the operators that take prompts in and verify trees of drafted tokens.

Five operators: attention over whole prompts or chunks of them (``prompt_attention``), attention of trees of drafted
tokens over a cache (``draft_attention``), the drafts that stand (``accept_drafts``), their keys and values moved
together (``keep_drafts``), and log probabilities of given tokens with entropy and top alternatives
(``token_logprobs``).  Each has a plain form in elementary torch operations, here, and, where numbers are computed, a
form in 64 bits (``exact``) written apart from it.  Page pools are those of this package: ``[page][kv head][16][d]``.
"""
import math

import torch

own = False

PAGE = 16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt, alone: latency
        dict(name="prompt short", op="prompt", requests=1, new_from=75, new_to=75, held_from=0, held_to=0, heads=32,
             kv_heads=8, d=128, dtype="bf16"),
        # prompts of very different lengths, packed
        dict(name="prompt packed", op="prompt", requests=24, new_from=60, new_to=2000, held_from=0, held_to=0, heads=32,
             kv_heads=8, d=128, dtype="bf16"),
        # one chunk each of three long documents, behind what earlier chunks left
        dict(name="prompt chunk", op="prompt", requests=3, new_from=2000, new_to=2048, held_from=3000, held_to=30000,
             heads=64, kv_heads=8, d=128, dtype="fp16"),
        # one long prompt at once
        dict(name="prompt long", op="prompt", requests=1, new_from=16384, new_to=16384, held_from=0, held_to=0, heads=64,
             kv_heads=8, d=128, dtype="bf16"),
        # the smallest tree of this repository with drafts: latency
        dict(name="drafts small", op="draft", requests=4, nodes=8, held_from=256, held_to=288, heads=4, kv_heads=4, d=64,
             dtype="bf16", ragged=False),
        # a mid-size batch; some requests have few drafts or sit the step out
        dict(name="drafts batch", op="draft", requests=64, nodes=26, held_from=500, held_to=4000, heads=32, kv_heads=8,
             d=128, dtype="bf16", ragged=True),
        # large trees behind long contexts
        dict(name="drafts long", op="draft", requests=16, nodes=60, held_from=8000, held_to=32000, heads=64, kv_heads=8,
             d=128, dtype="fp16", ragged=False),
        # the token just drawn, with five alternatives: one row, latency
        dict(name="scores one", op="scores", rows=1, vocab=32000, stride=32000, tokens=1, top=5, dtype="fp32",
             temperature=False),
        # every node of a batch of draft trees: the drafted token's probability and the eight children to grow
        dict(name="scores drafts", op="scores", rows=1664, vocab=50257, stride=50304, tokens=1, top=8, dtype="bf16",
             temperature=True),
        # the tokens of a prompt scored
        dict(name="scores prompt", op="scores", rows=2048, vocab=128000, stride=128000, tokens=1, top=0, dtype="fp32",
             temperature=False),
        # few small trees, one layer: latency
        dict(name="accept small", op="accept", requests=4, nodes=8, held=40, kv_heads=4, d=64, layers=1, dtype="bf16",
             ragged=False),
        # a batch of large trees, the pools of all layers
        dict(name="accept batch", op="accept", requests=64, nodes=60, held=200, kv_heads=8, d=128, layers=16,
             dtype="bf16", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


_HEADS = [(4, 4), (32, 32), (32, 8), (64, 8), (28, 4), (24, 8), (8, 1), (40, 8), (16, 2)]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "draft", "draft", "scores", "scores", "accept"])
    if op == "prompt":
        hq, hkv = rng.choice(_HEADS)
        new = _log(rng, 1, 8000)
        held = rng.choice([0, 0, _log(rng, 1, 30000)])
        most = int(min(16384 * 16384 * 64 // hq, 3000000000 // (hq // hkv)) // (new * (new + held)))
        return dict(op=op, requests=_log(rng, 1, max(1, min(200, most, 40000 // new, 400000 // (new + held)))),
                    new_from=_log(rng, 1, new), new_to=new, held_from=min(held, _log(rng, 1, max(1, held))), held_to=held,
                    heads=hq, kv_heads=hkv, d=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "draft":
        hq, hkv = rng.choice(_HEADS)
        n = rng.choice([1, _log(rng, 1, 128), _log(rng, 2, 64)])
        held = _log(rng, 1, 32000)
        return dict(op=op, requests=_log(rng, 1, max(1, min(512, 4000000 // (held * hkv), 500000000 // (n * hq * held)))),
                    nodes=n, held_from=_log(rng, 1, held), held_to=held, heads=hq, kv_heads=hkv,
                    d=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "bf16", "fp16"]), ragged=rng.random() < 0.6)
    if op == "scores":
        v = _log(rng, 700, 200000)
        return dict(op=op, rows=_log(rng, 1, max(1, min(8000, 200000000 // v))), vocab=v, stride=v + rng.choice([0, 0, 1, 40]),
                    tokens=rng.choice([1, 1, 3]), top=rng.choice([0, 1, 5, 8, 20, 64]), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                    temperature=rng.random() < 0.5)
    n = _log(rng, 1, 128)
    b = _log(rng, 1, max(1, min(512, 8000 // n)))
    h = rng.choice([1, 2, 4, 5, 8])
    return dict(op=op, requests=b, nodes=n, held=_log(rng, 1, 300), kv_heads=h, d=rng.choice([64, 128]),
                layers=_log(rng, 1, max(1, min(40, 8000 // (b * h)))), dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"op": case["op"], **globals()["_prepare_" + case["op"]](case, g)}


def _ints(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")


def _spread(g, n, lo, hi):
    """Whole numbers from lo to hi, spread over their logarithm, in any order: the same ones for every seed."""
    at = (torch.randperm(n, generator=g, device="cuda").double() + 0.5) / n
    return (torch.exp(math.log(lo + 1) + at * (math.log(hi + 1) - math.log(lo + 1))).round().long() - 1).clamp(lo, hi)


def _tables(g, lens, most, total=None):
    """Pages in shuffled order (out of `total`) for requests of these lengths; how many there are."""
    pages = (lens + PAGE - 1) // PAGE
    total = int(pages.sum()) if total is None else total
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first, column = torch.cumsum(pages, 0) - pages, torch.arange(max(1, (most + PAGE - 1) // PAGE), device="cuda")
    table = torch.where(column < pages[:, None], order[(first[:, None] + column).clamp(max=max(total - 1, 0))] if total else -1, -1)
    return table.to(torch.int32).contiguous(), max(total, 1)


def _trees(g, n, tokens):
    """Parents (within each request; node 0 is the root) and drafted tokens for n[b] nodes a request, and offsets."""
    cu = torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])
    t = torch.arange(tokens, device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=n.numel() - 1)
    node = t - cu[r]
    shape = torch.rand((tokens,), generator=g, device="cuda", dtype=torch.float64)
    # many children near the root, some deep chains
    parent = torch.where(node > 0, torch.where(shape < 0.3, node - 1, (node * ((shape - 0.3) / 0.7) ** 1.5).long()), -1)
    parent = torch.minimum(parent, node - 1)
    drafted = torch.randint(0, 32000, (tokens,), generator=g, device="cuda")
    return parent.to(torch.int32), drafted.to(torch.int32), cu.to(torch.int32), r, t < cu[-1]


def _pool(g, shape, kind):
    return torch.randn(shape, generator=g, device="cuda", dtype=kind)


def _prepare_prompt(c, g):
    b, hq, hkv, d, kind = c["requests"], c["heads"], c["kv_heads"], c["d"], TYPES[c["dtype"]]
    n, held = _spread(g, b, c["new_from"], c["new_to"]), _spread(g, b, c["held_from"], c["held_to"])
    lens = held + n
    table, total = _tables(g, lens, c["new_to"] + c["held_to"])
    tokens = int(n.sum())
    q = _pool(g, (tokens, hq + 2 * hkv, d), kind)[:, :hq]  # the queries' part of a joint projection
    cu = torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])
    return dict(q=q, k=_pool(g, (total, hkv, PAGE, d), kind), v=_pool(g, (total, hkv, PAGE, d), kind), table=table,
                lens=lens.to(torch.int32), cu=cu.to(torch.int32), most_new=c["new_to"], parents=None)


def _prepare_draft(c, g):
    b, hq, hkv, d, kind = c["requests"], c["heads"], c["kv_heads"], c["d"], TYPES[c["dtype"]]
    n = _ints(g, b, 0, c["nodes"]) if c["ragged"] else torch.full((b,), c["nodes"], device="cuda")
    lens = _spread(g, b, c["held_from"], c["held_to"]) + n
    table, total = _tables(g, lens, c["held_to"] + c["nodes"])
    tokens = b * c["nodes"]  # as many as a captured step has room for: those behind the last request's are padding
    parents, _, cu, _, _ = _trees(g, n, tokens)
    q = _pool(g, (tokens, hq + 2 * hkv, d), kind)[:, :hq]
    return dict(q=q, k=_pool(g, (total, hkv, PAGE, d), kind), v=_pool(g, (total, hkv, PAGE, d), kind), table=table,
                lens=lens.to(torch.int32), cu=cu, most_new=c["nodes"], parents=parents)


def _prepare_scores(c, g):
    r, v = c["rows"], c["vocab"]
    # a broad bulk and some tens of likely tokens a row
    x = torch.randn((r, c["stride"]), generator=g, device="cuda").mul_(2.2)
    likely = torch.randint(0, v, (r, 60), generator=g, device="cuda")
    x.scatter_add_(1, likely, 9 * torch.rand((r, 60), generator=g, device="cuda"))
    if r >= 8:
        x[1, : v // 2] = -math.inf  # a grammar's mask
        x[2, :v] = -math.inf  # one that leaves nothing
    tokens = torch.where(torch.rand((r, c["tokens"]), generator=g, device="cuda") < 0.7, likely[:, : c["tokens"]],
                         torch.randint(0, v, (r, c["tokens"]), generator=g, device="cuda")).to(torch.int32)
    if r >= 8:
        tokens[5, 0] = -1  # a place that has none
    temperature = 0.6 + 0.7 * torch.rand((r,), generator=g, device="cuda") if c["temperature"] else None
    return dict(logits=x.to(TYPES[c["dtype"]])[:, :v], tokens=tokens, temperature=temperature, top=c["top"])


def _prepare_accept(c, g):
    b, hkv, d, kind = c["requests"], c["kv_heads"], c["d"], TYPES[c["dtype"]]
    n = _ints(g, b, 0, c["nodes"]) if c["ragged"] else torch.full((b,), c["nodes"], device="cuda")
    lens = _ints(g, b, c["held"] // 2, c["held"]) + n
    table, total = _tables(g, lens, c["held"] + c["nodes"], b * ((c["held"] + c["nodes"] + PAGE - 1) // PAGE))
    tokens = b * c["nodes"]
    parents, drafted, cu, r, there = _trees(g, n, tokens)
    # at three nodes of four the target draws what the first child holds
    t = torch.arange(tokens, device="cuda")
    parent = torch.where(there & (parents >= 0), cu[r].long() + parents, tokens)
    first = torch.full((tokens + 1,), tokens, device="cuda").scatter_reduce(0, parent, t, "amin")[:-1]
    other = torch.randint(0, 32000, (tokens,), generator=g, device="cuda").to(torch.int32)
    child = drafted[first.clamp(max=tokens - 1)]
    stands = (first < tokens) & (torch.rand((tokens,), generator=g, device="cuda") < 0.75)
    pool = lambda: _pool(g, (c["layers"], total, hkv, PAGE, d), kind)  # noqa: E731
    return dict(drafted=drafted, parents=parents, cu=cu, sampled=torch.where(stands, child, other), table=table,
                lens=lens.to(torch.int32), k=pool(), v=pool(), most_new=c["nodes"])


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["op"]
    if own:
        import tree_structured_decode_gb300 as ta

        if op == "prompt":
            return ta.prompt_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"])
        if op == "draft":
            return ta.draft_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["parents"], s["cu"])
        if op == "scores":
            out = ta.token_logprobs(s["logits"], s["tokens"], temperature=1.0 if s["temperature"] is None else s["temperature"],
                                    top=s["top"])
            return out if s["top"] else out[:2]
        path, kept, token, back = ta.accept_drafts(s["drafted"], s["parents"], s["cu"], s["sampled"])
        ta.keep_drafts(path, s["cu"], s["table"], s["lens"], s["k"], s["v"])
        return path, kept, token, back, s["k"], s["v"]
    return _plain_attention(s) if op in ("prompt", "draft") else globals()["_plain_" + op](s)


def _ancestors(parent):
    """[.., n, n] truth values: whether j is i or above it, from parents [.., n] (-1: none), by doubling."""
    n = parent.shape[-1]
    node = torch.arange(n + 1, device=parent.device)
    up = torch.cat([torch.where(parent < 0, n, parent), torch.full_like(parent[..., :1], n)], -1)  # n: above every root
    seen = (node == node[:, None]).expand(*parent.shape[:-1], n + 1, n + 1)
    for _ in range(max(1, n).bit_length()):
        seen = seen | torch.take_along_dim(seen, up[..., None], -2)
        up = torch.take_along_dim(up, up, -1)
    return seen[..., :n, :n]


def _plain_attention(s):
    q, k, v, lens, table = s["q"], s["k"], s["v"], s["lens"].long(), s["table"].long()
    t, hq, d = q.shape
    hkv, b, most = k.shape[1], lens.numel(), s["most_new"]
    g, cu = hq // hkv, s["cu"].long()
    n = cu[1:] - cu[:-1]
    token = torch.arange(t, device=q.device)
    r = torch.searchsorted(cu[1:], token, right=True)  # b for padding, which sees nothing
    there = r < b
    rb = r.clamp(max=b - 1)
    j = torch.where(there, token - cu[rb], 0)
    key = torch.arange(table.shape[1] * PAGE, device=q.device)
    base = lens - n
    if s["parents"] is None:
        hidden = key > (base[:, None] + torch.arange(most, device=q.device))[:, :, None]  # [b, most, keys]
    else:
        parent = torch.full((b + 1, most), -1, device=q.device)
        parent[r, j] = s["parents"].long()
        sees = _ancestors(parent[:b])
        at = (key - base[:, None]).clamp(0, most - 1)
        hidden = ~torch.take_along_dim(sees, at[:, None, :].expand(b, most, -1), -1)
        hidden &= key >= base[:, None, None]
        hidden |= (key >= lens[:, None])[:, None]
    out, lse = torch.zeros((t, hq, d), device=q.device, dtype=q.dtype), torch.full((t, hq), -math.inf, device=q.device)
    for h in range(hkv):  # the scores of one kv head at a time fit the memory
        keys = k[:, h][table.clamp(min=0)].reshape(b, -1, d).float()
        values = v[:, h][table.clamp(min=0)].reshape(b, -1, d).float()
        qp = torch.zeros((b + 1, most, g, d), device=q.device)
        qp[r, j] = torch.where(there[:, None, None], q[:, h * g : (h + 1) * g].float() * (1 / math.sqrt(d)), 0)
        x = torch.matmul(qp[:b].reshape(b, most * g, d), keys.transpose(1, 2)).view(b, most, g, -1)
        x.masked_fill_(hidden[:, :, None], -math.inf)
        top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
        x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x.view(b, most * g, -1), values).view(b, most, g, d) / total.clamp(min=1e-30)
        there_h = there[:, None]
        out[:, h * g : (h + 1) * g] = torch.where(there_h[:, :, None], o[rb, j], 0).to(q.dtype)
        lse[:, h * g : (h + 1) * g] = torch.where(there_h, (top + total.log())[rb, j, :, 0], -math.inf)
        del x
    return out, lse


def _plain_scores(s):
    x = s["logits"].float()
    v, top, tokens = x.shape[1], s["top"], s["tokens"].long()
    broken = (x.isnan().any(1) | (x.amax(1) == -math.inf))[:, None]
    most = x.amax(1, keepdim=True)
    y = (x - torch.where(broken, 0, most)).div_(1.0 if s["temperature"] is None else s["temperature"][:, None])
    w = y.exp()
    total = w.sum(1, keepdim=True)
    log = total.log()
    entropy = log[:, 0] - w.mul_(y.clamp(min=-1e30)).sum(1) / total[:, 0]
    entropy = torch.where(broken[:, 0], math.nan, entropy)
    given = torch.where((tokens >= 0) & (tokens < v) & ~broken, y.gather(1, tokens.clamp(0, v - 1)) - log, math.nan)
    if top == 0:
        return given, entropy
    value, at = torch.sort(x, dim=1, descending=True, stable=True)  # of equal ones the first
    at, value = at[:, :top], value[:, :top]
    best = torch.where(broken, math.nan, y.gather(1, at) - log)
    at = torch.where(broken | (value == -math.inf), -1, at).to(torch.int32)
    return given, entropy, at, best


def _plain_accept(s):
    parents, drafted, cu, sampled, lens, table = s["parents"].long(), s["drafted"], s["cu"].long(), s["sampled"], s["lens"].long(), s["table"].long()
    t, b, most, device = drafted.numel(), lens.numel(), s["most_new"], drafted.device
    n = cu[1:] - cu[:-1]
    token = torch.arange(t, device=device)
    r = torch.searchsorted(cu[1:], token, right=True)
    j = torch.where(r < b, token - cu[r.clamp(max=b - 1)], 0)
    # one row of nodes a request
    pad = lambda x, other: torch.full((b + 1, most), other, device=device).index_put_((r, j), x.long())[:b]  # noqa: E731
    parent, draft, drawn = pad(parents, -1), pad(drafted, -1), pad(sampled, -2)
    node = torch.arange(most, device=device)
    real = node < n[:, None]
    match = real & (node > 0) & (parent >= 0) & (draft == drawn.gather(1, parent.clamp(min=0))) & (draft >= 0)
    # of siblings that match, the first
    first = torch.full((b, most + 1), most, device=device)
    first = first.scatter_reduce(1, torch.where(match, parent, most), node.expand(b, most), "amin")
    match &= first.gather(1, parent.clamp(min=0)) == node
    # a node stands where it and all above it match
    top = torch.where(match, parent, -1)
    sees = _ancestors(top)
    stands = real & sees[:, :, 0]
    kept = stands.sum(1)
    order = torch.argsort((~stands).to(torch.int8), dim=1, stable=True)  # the path: those that stand, by index
    path = torch.where(node < kept[:, None], order, -1)
    last = path.gather(1, (kept - 1).clamp(min=0)[:, None]).clamp(min=0)
    following = torch.where(kept > 0, drawn.gather(1, last)[:, 0], -1)
    flat = torch.where(r < b, path[r.clamp(max=b - 1), j], -1)
    # the keys and values of those that stand, to the places behind what is held
    held = (lens - n)[:, None]
    here, row = node < kept[:, None], torch.arange(b, device=device)[:, None].expand(b, most)
    rows, source, target = row[here], (held + path)[here], (held + node)[here]
    from_page, to_page = table[rows, source // PAGE], table[rows, target // PAGE]
    s["k"][:, to_page, :, target % PAGE] = s["k"][:, from_page, :, source % PAGE]
    s["v"][:, to_page, :, target % PAGE] = s["v"][:, from_page, :, source % PAGE]
    return flat.to(torch.int32), kept.to(torch.int32), following.to(torch.int32), (kept - n).to(torch.int32), s["k"], s["v"]


# ------------------------------------------------------------------ what a pass cannot do without
def _mean(lo, hi):
    return lo if hi == lo else (hi - lo) / math.log((hi + 1) / (lo + 1)) - 1


def work(case):
    c = case
    if c["op"] in ("prompt", "draft"):
        if c["op"] == "prompt":
            n, held = _mean(c["new_from"], c["new_to"]), _mean(c["held_from"], c["held_to"])
            lo, hi = c["new_from"], c["new_to"]  # the mean of n^2 under the same spread
            square = lo * lo if hi == lo else (hi * hi - lo * lo) / 2 / math.log((hi + 1) / (lo + 1))
            pairs = c["requests"] * (n * held + square / 2 + n / 2)
        else:
            n, held = c["nodes"] / 2 if c["ragged"] else c["nodes"], _mean(c["held_from"], c["held_to"])
            pairs = c["requests"] * n * (held + 1 + math.log(1 + n))
        t = c["requests"] * n
        kv = c["requests"] * (held + n) * 2 * c["kv_heads"] * c["d"] * 2
        return {"bytes": kv + t * c["heads"] * (c["d"] * 4 + 4), "flops": 4.0 * c["d"] * c["heads"] * pairs}
    if c["op"] == "scores":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": float(c["rows"]) * (c["vocab"] * size + 8 * c["tokens"] + 8 * c["top"] + 8), "flops": 5.0 * c["rows"] * c["vocab"]}
    nodes = c["requests"] * (c["nodes"] / 2 if c["ragged"] else c["nodes"])
    moved = c["requests"] * min(2.0, c["nodes"] / 4)  # about two drafts a request are kept and not in place already
    return {"bytes": 16.0 * nodes + 4 * c["requests"] + moved * c["layers"] * 2 * 2 * c["kv_heads"] * c["d"] * 2, "flops": 0.0}


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    if case["op"] == "accept":
        return None  # whole numbers and copies
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    return _exact_attention(s) if case["op"] in ("prompt", "draft") else _exact_scores(s)


def _exact_attention(s):
    """Request by request, kv head by kv head, a few rows at a time."""
    q, k, v = s["q"], s["k"], s["v"]
    (t, hq, d), hkv = q.shape, k.shape[1]
    g = hq // hkv
    out = torch.zeros((t, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((t, hq), -math.inf, dtype=torch.float64, device=q.device)
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    parents = None if s["parents"] is None else s["parents"].tolist()
    for i, length in enumerate(lens):
        n = cu[i + 1] - cu[i]
        if n == 0:
            continue
        held, pages = length - n, s["table"][i, : (length + PAGE - 1) // PAGE].long()
        if parents is None:
            see = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
        else:
            above = [[] for _ in range(n)]
            for a in range(n):
                up = parents[cu[i] + a]
                above[a] = [a] + (above[up] if up >= 0 else [])
            see = torch.tensor([[x in row for x in range(n)] for row in map(set, above)], device=q.device)
        for h in range(hkv):
            keys, values = k[pages, h].reshape(-1, d)[:length].double(), v[pages, h].reshape(-1, d)[:length].double()
            step = max(1, 200_000_000 // (g * length))
            for a in range(0, n, step):
                z = min(n, a + step)
                x = torch.einsum("ngd,ld->ngl", q[cu[i] + a : cu[i] + z, h * g : (h + 1) * g].double(), keys) / math.sqrt(d)
                x[:, :, held:].masked_fill_(~see[a:z, None], -math.inf)
                part = torch.logsumexp(x, -1)
                lse[cu[i] + a : cu[i] + z, h * g : (h + 1) * g] = part
                out[cu[i] + a : cu[i] + z, h * g : (h + 1) * g] = (x - part[..., None]).exp() @ values
    return out, lse


def _exact_scores(s):
    """Some rows at a time, by logsumexp; probabilities p give the entropy as -sum p ln p."""
    given, entropy, best = [], [], []
    for a in range(0, s["logits"].shape[0], 64):
        x = s["logits"][a : a + 64].double()
        if s["temperature"] is not None:
            x = x / s["temperature"][a : a + 64, None].double()
        broken = x.isnan().any(1) | ~(x > -math.inf).any(1)
        log_p = x - torch.logsumexp(x, 1, keepdim=True)
        log_p[broken] = math.nan
        p = log_p.exp()
        entropy.append(-torch.where(p > 0, p * log_p, p).sum(1))
        tokens = s["tokens"][a : a + 64].long()
        fine = (tokens >= 0) & (tokens < x.shape[1])
        given.append(torch.where(fine, log_p.gather(1, tokens.clamp(0, x.shape[1] - 1)), math.nan))
        best.append(torch.where(broken[:, None], math.nan, torch.topk(log_p.nan_to_num(0.0, neginf=-math.inf), s["top"], dim=1).values))
    return torch.cat(given), torch.cat(entropy), *((None, torch.cat(best)) if s["top"] else ())
