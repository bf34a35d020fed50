"""Cases for the operators of a decode loop whose lengths live on the GPU.

Four operators: the page tables and slot maps of a batch (``extend_tables``), the append of new keys and values by
slot (``append_slots``), attention of a batch whose requests share a long prefix (``prefix_attention``) and sampling
from given random numbers (``sample``).  Each has a plain form in elementary torch operations, here, and a form in
64 bits (``exact``) written apart from it.  Layouts are those of the page pools of this package: K and V pages
``[page][kv head][16][d]``.
"""
import math

import torch

own = False

PAGE = 16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a mid-size batch: one token a request, a new page now and then; latency is all that counts
        dict(name="tables decode", op="tables", requests=256, held=2000, new=1, ragged=False),
        # a batch of prompts taken in at once: every page and slot of up to 2048 tokens a request
        dict(name="tables prompts", op="tables", requests=64, held=0, new=2048, ragged=True),
        # the new tokens of one decode step of 256 requests, 8 kv heads
        dict(name="append decode", op="append", tokens=256, padding=0, kv_heads=8, d=128, dtype="bf16"),
        # the keys and values of a chunk of prompts, with the padding that a fixed-size batch has
        dict(name="append prompts", op="append", tokens=16384, padding=411, kv_heads=8, d=128, dtype="bf16"),
        # the smallest tree of this repository: 4 requests behind 256 tokens, latency
        dict(name="attend tiny", op="attend", requests=4, heads=4, kv_heads=4, d=64, prefix=256, own_from=32,
             own_to=32, new=1, dtype="bf16"),
        # long prompt, few requests, no sharing of kv heads: splitting the prefix over the GPU
        dict(name="attend long", op="attend", requests=10, heads=32, kv_heads=32, d=128, prefix=4000, own_from=380,
             own_to=420, new=1, dtype="bf16"),
        # many samples of one prompt, early in their answers
        dict(name="attend wide", op="attend", requests=256, heads=32, kv_heads=8, d=128, prefix=2048, own_from=50,
             own_to=80, new=1, dtype="bf16"),
        # up to 4 speculative tokens a request (some requests sit a step out), very uneven lengths, a prefix that ends inside a page
        dict(name="attend drafts", op="attend", requests=128, heads=64, kv_heads=4, d=128, prefix=5003, own_from=16,
             own_to=2048, new=4, dtype="fp16"),
        # a large batch behind a long shared document
        dict(name="attend document", op="attend", requests=512, heads=64, kv_heads=8, d=128, prefix=32768, own_from=16,
             own_to=1024, new=1, dtype="bf16"),
        # one request, one token
        dict(name="sample one", op="sample", rows=1, vocab=32000, stride=32000, draws=1, dtype="fp32", filters="all"),
        # a batch in 16 bits with every filter, an odd vocabulary in a padded buffer, four branches drawn from each row
        dict(name="sample branches", op="sample", rows=128, vocab=50257, stride=50304, draws=4, dtype="bf16",
             filters="all"),
        # a large batch and vocabulary, top-p alone: the sums go over whole rows
        dict(name="sample large", op="sample", rows=256, vocab=128000, stride=128000, draws=1, dtype="fp32",
             filters="top_p"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "sample", "sample"])
    if op == "tables":
        b = _log(rng, 1, 2000)
        return dict(op=op, requests=b, held=rng.choice([0, _log(rng, 1, 4000)]),
                    new=_log(rng, 1, max(1, min(2048, 120000 // b))), ragged=rng.random() < 0.6)
    if op == "append":
        n = _log(rng, 1, 16000)
        return dict(op=op, tokens=n, padding=rng.choice([0, 1, n // 7]), kv_heads=rng.choice([1, 2, 4, 5, 8]),
                    d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "fp16"]))
    if op == "attend":
        hq, hkv = rng.choice([(4, 4), (32, 32), (32, 8), (64, 4), (64, 8), (28, 4), (24, 8), (8, 1), (40, 8)])
        new = rng.choice([1, 1, 1, 2, 4, 5])
        own_to = _log(rng, new, 2000)
        return dict(op=op, requests=_log(rng, 1, max(1, min(512, 4000000 // (own_to * hkv * new), 2048 // new))), heads=hq,
                    kv_heads=hkv, d=rng.choice([64, 128, 128]), prefix=rng.choice([0, _log(rng, 1, 32000 // new)]),
                    own_from=_log(rng, new, own_to), own_to=own_to, new=new, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    v = _log(rng, 900, 128000)
    return dict(op=op, rows=_log(rng, 1, 250), vocab=v, stride=v + rng.choice([0, 0, 1, 40]), draws=rng.choice([1, 1, 2, 5]),
                dtype=rng.choice(["fp32", "bf16", "fp16"]), filters=rng.choice(["all", "none", "top_k", "top_p", "min_p"]))


# ------------------------------------------------------------------ inputs
def _ints(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"op": case["op"], **globals()["_prepare_" + case["op"]](case, g)}


def _prepare_tables(c, g):
    b = c["requests"]
    held = _ints(g, b, c["held"] // 2, c["held"]) if c["held"] else torch.zeros(b, dtype=torch.int64, device="cuda")
    new = _ints(g, b, 1, c["new"]) if c["ragged"] else torch.full((b,), c["new"], device="cuda")
    width = (c["held"] + c["new"] + PAGE - 1) // PAGE + 1
    # pages in shuffled order: first those that the requests hold, then the stack of free ones
    held_pages = (held + PAGE - 1) // PAGE
    total = b * width
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(held_pages, 0) - held_pages
    column = torch.arange(width, device="cuda")
    table = torch.where(column < held_pages[:, None], order[(first[:, None] + column).clamp(max=total - 1)], -1).to(torch.int32)
    used = held_pages.sum()
    return dict(lens=held.to(torch.int32), new=new.to(torch.int32), back=-new.to(torch.int32), table=table.contiguous(),
                free=torch.roll(order, -int(used)).contiguous(), n_free=(total - used).to(torch.int32).reshape(1),
                most=b * c["new"], base=1000)


def _prepare_append(c, g):
    t, h, d, kind = c["tokens"], c["kv_heads"], c["d"], TYPES[c["dtype"]]
    pages = max(1, 2 * (t + PAGE - 1) // PAGE)
    pool = lambda: torch.randn((pages, h, PAGE, d), generator=g, device="cuda", dtype=kind)  # noqa: E731
    both = torch.randn((t, 2, h, d), generator=g, device="cuda", dtype=kind)  # K and V of a token side by side, as one projection gives them
    slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:t].to(torch.int32)
    if c["padding"]:
        slots[-c["padding"]:] = -1
    return dict(k_new=both[:, 0], v_new=both[:, 1], slots=slots, k=pool(), v=pool())


def _prepare_attend(c, g):
    b, hq, hkv, d, kind = c["requests"], c["heads"], c["kv_heads"], c["d"], TYPES[c["dtype"]]
    span = torch.rand((b,), generator=g, device="cuda", dtype=torch.float64)
    lens = torch.exp(math.log(c["own_from"]) + span * (math.log(c["own_to"]) - math.log(c["own_from"]))).round().to(torch.int64)
    lens = lens.clamp(c["own_from"], c["own_to"])
    n = torch.full((b,), 1, device="cuda") if c["new"] == 1 else _ints(g, b, 0, c["new"])
    cu = torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])
    tokens = b * c["new"]  # as many as a captured step has room for: those behind the last request's are padding
    np_ = (lens + PAGE - 1) // PAGE
    width = (c["own_to"] + PAGE - 1) // PAGE
    pre = (c["prefix"] + PAGE - 1) // PAGE
    total = pre + int(np_.sum())
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = pre + torch.cumsum(np_, 0) - np_
    column = torch.arange(width, device="cuda")
    table = torch.where(column < np_[:, None], order[(first[:, None] + column).clamp(max=total - 1)], -1).to(torch.int32)
    pool = lambda: torch.randn((total, hkv, PAGE, d), generator=g, device="cuda", dtype=kind)  # noqa: E731
    q = torch.randn((tokens, hq + 2 * hkv, d), generator=g, device="cuda", dtype=kind)[:, :hq]  # the queries' part of a joint projection
    return dict(q=q, k=pool(), v=pool(), prefix_pages=order[:pre].contiguous(), prefix=c["prefix"], table=table.contiguous(),
                lens=lens.to(torch.int32), cu=None if c["new"] == 1 else cu.to(torch.int32), most_new=c["new"])


def _prepare_sample(c, g):
    r, v = c["rows"], c["vocab"]
    # a broad bulk and some tens of likely tokens a row
    x = torch.randn((r, c["stride"]), generator=g, device="cuda").mul_(2.2)
    likely = torch.randint(0, v, (r, 60), generator=g, device="cuda")
    x.scatter_add_(1, likely, 9 * torch.rand((r, 60), generator=g, device="cuda"))
    if r >= 8:
        x[1, : v // 2] = -math.inf  # a grammar's mask
        x[2, :v] = -math.inf  # one that leaves nothing
    logits = x.to(TYPES[c["dtype"]])[:, :v]
    f = c["filters"]
    temperature = 0.6 + 0.7 * torch.rand((r,), generator=g, device="cuda")
    if r >= 8:
        temperature[3] = 0  # greedy
    top_k = _ints(g, r, 1, min(v, 400)).to(torch.int32) if f in ("all", "top_k") else None
    top_p = 0.7 + 0.3 * torch.rand((r,), generator=g, device="cuda") if f in ("all", "top_p") else None
    min_p = 0.1 * torch.rand((r,), generator=g, device="cuda") if f in ("all", "min_p") else None
    return dict(logits=logits, u=torch.rand((r, c["draws"]), generator=g, device="cuda"), temperature=temperature, top_k=top_k,
                top_p=top_p, min_p=min_p)


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["op"]
    if own:
        import tree_structured_decode_gb300 as ta

        s = state
        if op == "tables":
            # a step's extension, and its tokens taken back (drafts that were rejected, requests that ended): the state is as before
            out = ta.extend_tables(s["lens"], s["new"], s["table"], s["free"], s["n_free"], s["most"], position_base=s["base"])
            ta.extend_tables(s["lens"], s["back"], s["table"], s["free"], s["n_free"], 0)
            return *out, s["lens"], s["table"], s["free"], s["n_free"]
        if op == "append":
            ta.append_slots(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"])
            return s["k"], s["v"]
        if op == "attend":
            return ta.prefix_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["prefix_pages"], s["prefix"])
        return ta.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    return globals()["_plain_" + op](state)


def _plain_extend(lens, new, table, free, n_free, most, base):
    """lens, table, free and n_free are changed in place; the tables always suffice here."""
    n, held = new.long(), lens.long()
    after = (held + n).clamp(min=0)
    old, now = (held + PAGE - 1) // PAGE, (after + PAGE - 1) // PAGE
    need, back = (now - old).clamp(min=0), (old - now).clamp(min=0)
    first_need, first_back = torch.cumsum(need, 0) - need, torch.cumsum(back, 0) - back
    column = torch.arange(table.shape[1], device=table.device)
    stack = n_free.long()
    # new pages come from the top of the stack
    at = stack - 1 - (first_need[:, None] + column - old[:, None])
    taken = (column >= old[:, None]) & (column < now[:, None])
    table.copy_(torch.where(taken, free[at.clamp(0, free.numel() - 1)], table))
    # pages given back: the last one lowest, so that what was just taken lies as before
    stack = stack - need.sum()
    at = stack + back.sum() - 1 - (first_back[:, None] + column - now[:, None])
    given = (column >= now[:, None]) & (column < old[:, None])
    spare = torch.cat([free, free.new_zeros(1)])
    spare.scatter_(0, torch.where(given, at, free.numel()).reshape(-1), table.reshape(-1))
    free.copy_(spare[:-1])
    # slots and positions of the new tokens
    add = n.clamp(min=0)
    cu = torch.cat([add.new_zeros(1), torch.cumsum(add, 0)])
    t = torch.arange(most, device=table.device)
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=n.numel() - 1)
    there = t < cu[-1]
    pos = held[r] + t - cu[r]
    page = table[r, (pos // PAGE).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(there, page * PAGE + pos % PAGE, -1).to(torch.int32)
    positions = torch.where(there, pos + base, -1).to(torch.int32)
    lens.copy_(after)
    n_free.copy_(stack + back.sum())
    return slots, positions, cu.to(torch.int32)


def _plain_tables(s):
    out = _plain_extend(s["lens"], s["new"], s["table"], s["free"], s["n_free"], s["most"], s["base"])
    _plain_extend(s["lens"], s["back"], s["table"], s["free"], s["n_free"], 0, 0)
    return *out, s["lens"], s["table"], s["free"], s["n_free"]


def _plain_append(s):
    there = s["slots"] >= 0
    at = s["slots"][there].long()
    s["k"][at // PAGE, :, at % PAGE] = s["k_new"][there]
    s["v"][at // PAGE, :, at % PAGE] = s["v_new"][there]
    return s["k"], s["v"]


def _plain_attend(s):
    q, k, v, lens, table = s["q"], s["k"], s["v"], s["lens"].long(), s["table"].long()
    t, hq, d = q.shape
    hkv, b, most = k.shape[1], lens.numel(), s["most_new"]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(b + 1, device=q.device)
    n = cu[1:] - cu[:-1]
    token = torch.arange(t, device=q.device)
    r = torch.searchsorted(cu[1:], token, right=True)  # b for padding, which sees nothing
    there = r < b
    j = torch.where(there, token - cu[r], 0)
    lens, n = torch.cat([lens, lens.new_zeros(1)]), torch.cat([n, n.new_ones(1)])
    qf = q.float().reshape(t, hkv, hq // hkv, d) * (1 / math.sqrt(d))
    pk = k[s["prefix_pages"].long()].float().transpose(0, 1).reshape(hkv, -1, d)[:, : s["prefix"]]
    pv = v[s["prefix_pages"].long()].float().transpose(0, 1).reshape(hkv, -1, d)[:, : s["prefix"]]
    before = torch.einsum("thgd,hld->thgl", qf, pk).masked_fill_(~there[:, None, None, None], -math.inf)
    # each request's own keys and values, padded to the longest
    ok = k[table.clamp(min=0)].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    ov = v[table.clamp(min=0)].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    qp = qf.new_zeros(b + 1, most, hkv, hq // hkv, d)
    qp[r, j] = qf
    rb = r.clamp(max=b - 1)
    after = torch.einsum("bnhgd,bhld->bnhgl", qp[:b], ok)[rb, j]
    end = torch.where(there, lens[r] - n[r] + j + 1, 0)
    after.masked_fill_((torch.arange(after.shape[-1], device=q.device) >= end[:, None])[:, None, None], -math.inf)
    top = torch.cat([before, after], -1).amax(-1, keepdim=True)
    shift = torch.where(top == -math.inf, torch.zeros_like(top), top)
    before, after = (before - shift).exp_(), (after - shift).exp_()
    total = before.sum(-1, keepdim=True) + after.sum(-1, keepdim=True)
    wp = qf.new_zeros(b + 1, most, hkv, hq // hkv, after.shape[-1])
    wp[r, j] = after
    out = torch.einsum("thgl,hld->thgd", before, pv) + torch.einsum("bnhgl,bhld->bnhgd", wp[:b], ov)[rb, j]
    out = torch.where(total > 0, out / total, 0)
    return out.reshape(t, hq, d).to(q.dtype), (top + total.log()).reshape(t, hq)


def _plain_sample(s):
    # sums over whole rows and comparisons next to their borders decide which token comes: 64 bits
    x = s["logits"].float() + 0.0
    r, v = x.shape
    broken = x.isnan().any(1) | (x.amax(1) == -math.inf)
    top = x.amax(1, keepdim=True)
    same = x == top
    temperature = s["temperature"][:, None].double()
    greedy = ~(temperature > 0)
    w = torch.where(same, 0.0, x.double() - top.double()).div_(torch.where(greedy, 1.0, temperature)).exp_()
    w = torch.where(greedy, same.double(), w)
    _, at = torch.sort(x, dim=1, descending=True, stable=True)
    ws = w.gather(1, at)
    rank = torch.arange(v, device=x.device)
    keep = torch.where(greedy, rank == 0, rank >= 0)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    if s["top_p"] is not None:
        p = s["top_p"][:, None].double()
        c = (ws * keep).cumsum_(1)
        keep[:, 1:] &= (c[:, :-1] < p * c[:, -1:]) | (p >= 1)
    if s["min_p"] is not None:
        keep[:, 1:] &= ws[:, 1:] >= s["min_p"][:, None].double()
    w = w * torch.zeros_like(keep).scatter_(1, at, keep)
    c = w.cumsum(1)
    total = c[:, -1:]
    token = torch.searchsorted(c, s["u"].double() * total, right=True).clamp(max=v - 1)
    logprob = (w.gather(1, token) / total).log().float()
    return torch.where(broken[:, None], -1, token).to(torch.int32), torch.where(broken[:, None], math.nan, logprob)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "tables":
        b = c["requests"]
        t = b * (c["new"] + 1) // 2 if c["ragged"] else b * c["new"]
        pages = t // PAGE + (b // 2 if c["ragged"] else 0)
        return {"bytes": 8.0 * b * c["new"] + 24.0 * b + 16.0 * pages, "flops": 0.0}  # slots, positions; lengths; pages out and back
    if c["op"] == "append":
        return {"bytes": (c["tokens"] - c["padding"]) * 2.0 * 2 * 2 * c["kv_heads"] * c["d"] + 4.0 * c["tokens"], "flops": 0.0}
    if c["op"] == "attend":
        lo, hi = c["own_from"], c["own_to"]
        mean = lo if hi == lo else (hi - lo) / math.log(hi / lo)
        t = c["requests"] * (1 if c["new"] == 1 else c["new"] / 2)
        kv = (c["prefix"] + c["requests"] * mean) * 2 * c["kv_heads"] * c["d"] * 2
        return {"bytes": kv + t * c["heads"] * (c["d"] * 4 + 4), "flops": 4.0 * c["d"] * c["heads"] * t * (c["prefix"] + mean)}
    size = 4 if c["dtype"] == "fp32" else 2
    return {"bytes": float(c["rows"]) * c["vocab"] * size + c["rows"] * (16 + 12.0 * c["draws"]), "flops": 4.0 * c["rows"] * c["vocab"]}


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "sample":
        return None, _exact_sample(s)
    return None  # whole numbers and copies


def _exact_attend(s):
    """Request by request and kv head by kv head: softmax attention over the prefix's and the request's own tokens, joined."""
    q, (t, hq, d) = s["q"].double(), s["q"].shape
    hkv, b = s["k"].shape[1], s["lens"].numel()
    g = hq // hkv
    if t * hq * d * (s["prefix"] + s["table"].shape[1] * PAGE) > 3e11:
        return None
    out, lse = torch.zeros_like(q), torch.full((t, hq), -math.inf, dtype=torch.float64, device=q.device)
    lens = s["lens"].tolist()
    cu = s["cu"].tolist() if s["cu"] is not None else list(range(b + 1))
    rows = lambda pool, pages, h, n: pool[pages.long(), h].double().reshape(-1, d)[:n]  # noqa: E731
    for h in range(hkv):
        kp, vp = rows(s["k"], s["prefix_pages"], h, s["prefix"]), rows(s["v"], s["prefix_pages"], h, s["prefix"])
        for i in range(b):
            n = cu[i + 1] - cu[i]
            if not n:
                continue
            pages = s["table"][i, : (lens[i] + PAGE - 1) // PAGE]
            keys = torch.cat([kp, rows(s["k"], pages, h, lens[i])])
            values = torch.cat([vp, rows(s["v"], pages, h, lens[i])])
            qi = q[cu[i] : cu[i + 1], h * g : (h + 1) * g].reshape(n * g, d)
            score = qi @ keys.T / math.sqrt(d)
            last = len(keys) - n + torch.arange(n, device=q.device).repeat_interleave(g)  # a draft does not see the drafts behind it
            score[torch.arange(len(keys), device=q.device)[None] > last[:, None]] = -math.inf
            z = torch.logsumexp(score, 1)
            out[cu[i] : cu[i + 1], h * g : (h + 1) * g] = (torch.exp(score - z[:, None]) @ values).reshape(n, g, d)
            lse[cu[i] : cu[i + 1], h * g : (h + 1) * g] = z.reshape(n, g)
    return out, lse


def _exact_sample(s):
    """Row by row on the host: the kept tokens' list, then the first whose sum passes u times the whole."""
    import numpy as np

    x = s["logits"].float().cpu().numpy().astype(np.float64)
    value = lambda name, i, other: other if s[name] is None else float(s[name][i])  # noqa: E731
    u = s["u"].double().cpu().numpy()
    got = np.full(u.shape, np.nan)
    for i, row in enumerate(x):
        if np.isnan(row).any() or row.max() == -np.inf:
            continue
        temperature, p = value("temperature", i, 1.0), value("top_p", i, 1.0)
        order = np.argsort(-row, kind="stable")
        if not temperature > 0:
            got[i] = 0.0
            continue
        part = np.exp((row[order] - row[order[0]]) / temperature)
        k = int(value("top_k", i, 0))
        size = min(k, row.size) if k > 0 else row.size
        if p < 1:
            size = min(size, 1 + int(np.searchsorted(np.cumsum(part[:size]), p * math.fsum(part[:size]), side="left")))
        size = max(1, min(size, int((part >= value("min_p", i, 0.0)).sum())))
        kept = np.sort(order[:size])
        sums = np.cumsum(np.exp((row[kept] - row[order[0]]) / temperature))
        pick = np.minimum(np.searchsorted(sums, u[i] * sums[-1], side="right"), size - 1)
        got[i] = (row[kept[pick]] - row[order[0]]) / temperature - math.log(sums[-1])
    return torch.from_numpy(got)
