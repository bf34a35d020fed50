"""Prompts taken in and drafts verified as a serving loop does it.

A captured step makes room for every node of the requests' trees, appends their
keys and values, attends, draws a token at every node, keeps the path that agrees,
moves its keys and values together and takes the rest back; it is replayed with
other trees and lengths, and after every replay each stage is compared with its
definition on what the stage before it gave."""
import numpy as np
import pytest
import torch

from oracle import batch as oracle_batch
from oracle import drafts as oracle
from test_chunk_attention import check as check_attention
from test_chunk_attention import tree

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu

ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy()  # noqa: E731


def test_a_captured_step_of_drafts_replayed():
    requests, most, hq, hkv, d, vocab, width, layers = 5, 9, 8, 2, 64, 7, 12, 2
    tokens = requests * most
    g = torch.Generator(device="cuda").manual_seed(2)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    pages = requests * width
    k, v = (randn(layers, pages, hkv, 16, d).to(torch.bfloat16) for _ in range(2))
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    n_free, lens, status = ints([pages]), ints([0] * requests), ints([0])
    table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    embed = randn(vocab, layers * (hq + 2 * hkv) * d).to(torch.bfloat16)
    head = 0.3 * randn(hq * d, vocab)
    u = torch.rand(tokens, generator=g, device="cuda")
    n_new, drafted, parents = ints([0] * requests), ints([0] * tokens), ints([-1] * tokens)
    stage = {}

    def step():
        slots, _, cu = ta.extend_tables(lens, n_new, table, free, n_free, tokens, status=status)
        x = embed[drafted.long()].reshape(tokens, layers, hq + 2 * hkv, d)
        outs = []
        for i in range(layers):
            y = x[:, i]
            ta.append_slots(y[:, hq:hq + hkv], y[:, hq + hkv:], slots, k[i], v[i], status=status)
            outs.append(ta.draft_attention(y[:, :hq], k[i], v[i], table, lens, parents, cu, status=status))
        logits = outs[-1][0].float().reshape(tokens, -1) @ head
        drawn, _ = ta.sample(logits, u)
        path, kept, following, back = ta.accept_drafts(drafted, parents, cu, drawn, status=status)
        stage.update(k=k.clone(), v=v.clone(), lens=lens.clone(), table=table.clone())
        ta.keep_drafts(path, cu, table, lens, k, v, status=status)
        ta.extend_tables(lens, back, table, free, n_free, 0, status=status)
        scores = ta.token_logprobs(logits, drawn, top=3)
        stage.update(x=x, outs=outs, logits=logits, drawn=drawn, path=path, kept=kept, following=following, back=back, cu=cu,
                     scores=scores)

    state = [t.clone() for t in (lens, table, free, n_free, k, v)]
    step()  # once outside a graph, and its state put back
    for t, was in zip((lens, table, free, n_free, k, v), state):
        t.copy_(was)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(3)
    held = [0] * requests
    for i in range(25):
        counts = [int(rng.integers(0, most + 1)) for _ in range(requests)]
        p = sum((tree(100 * i + b, n) for b, n in enumerate(counts)), [])
        # (several of a tree's roots but node 0 stand for nothing: all others hang below it)
        n_new.copy_(ints(counts))
        parents.copy_(ints(p + [-1] * (tokens - len(p))))
        drafted.copy_(ints(rng.integers(0, vocab, tokens).tolist()))
        u.copy_(torch.rand(tokens, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
        s = stage
        assert s["cu"].tolist() == cu
        assert s["lens"].tolist() == [h + n for h, n in zip(held, counts)]
        for layer in range(layers):
            check_attention(dict(q=s["x"][:, layer, :hq].cpu(), k=s["k"][layer].cpu(), v=s["v"][layer].cpu(), table=s["table"].cpu(),
                                 lens=s["lens"].cpu(), cu_all=np.array(cu), parents=parents.cpu(), dtype="bf16"), *s["outs"][layer])
        x, numbers, drawn = s["logits"].cpu().numpy(), u.cpu().numpy(), s["drawn"].tolist()
        for r in range(cu[-1]):
            assert drawn[r] == oracle_batch.sample(x[r], [numbers[r]])[0][0]
            want, entropy, best = oracle.token_logprobs(x[r], [drawn[r]], 1.0, 3)
            assert abs(s["scores"][0][r].item() - want[0]) <= 1e-5 and abs(s["scores"][1][r].item() - entropy) <= 1e-5
            assert s["scores"][2][r].tolist() == [t for t, _ in best]
        want = oracle.accept_drafts(drafted.tolist(), parents.tolist(), cu, drawn)
        assert [s[n].tolist() for n in ("path", "kept", "following", "back")] == list(want)
        kv = oracle.keep_drafts(want[0], cu, s["table"].cpu().numpy(), s["lens"].cpu().numpy(), bits(s["k"]), bits(s["v"]))
        assert np.array_equal(bits(k), kv[0]) and np.array_equal(bits(v), kv[1])
        held = [h + n for h, n in zip(held, want[1])]
        assert lens.tolist() == held
        if max(held) > 16 * width - 2 * most:  # the longest request ends
            back = [-h if h == max(held) else 0 for h in held]
            ta.extend_tables(lens, ints(back), table, free, n_free, 0, status=status)
            held = [h + x for h, x in zip(held, back)]
    assert status.item() == 0 and max(held) > 20


def test_a_prompt_in_chunks_and_the_tokens_behind_it():
    """A prompt taken in at once, in chunks, and its last token as a decode step: the same rows; single tokens as
    prefix_attention has them."""
    hq, hkv, d, length = 8, 2, 128, 700
    g = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x = randn(length, hq + 2 * hkv, d)
    k, v = randn(50, hkv, 16, d), randn(50, hkv, 16, d)
    free, n_free, lens = torch.randperm(50, generator=g, device="cuda").to(torch.int32), ints([50]), ints([0])
    table, rows = torch.full((1, 50), -1, dtype=torch.int32, device="cuda"), []
    for n in (128, 1, 300, 16, 255):
        at = sum(len(r) for r in rows)
        slots, _, cu = ta.extend_tables(lens, ints([n]), table, free, n_free, n)
        y = x[at:at + n]
        ta.append_slots(y[:, hq:hq + hkv], y[:, hq + hkv:], slots, k, v)
        rows.append(ta.prompt_attention(y[:, :hq], k, v, table, lens, cu)[0])
    whole, lse = ta.prompt_attention(x[:, :hq], k, v, table, lens, ints([0, length]))
    s = dict(q=x[:, :hq].cpu(), k=k.cpu(), v=v.cpu(), table=table.cpu(), lens=lens.cpu(), cu_all=np.array([0, length]), parents=None,
             dtype="bf16")
    check_attention(s, whole, lse)
    check_attention(s, torch.cat(rows), lse)
    one = ta.draft_attention(x[-1:, :hq], k, v, table, lens, ints([-1]))
    other = ta.prefix_attention(x[-1:, :hq], k, v, table, lens)
    s.update(q=s["q"][-1:], cu_all=np.array([0, 1]))
    check_attention(s, *one)
    check_attention(s, *other)
