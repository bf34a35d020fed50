"""The operators whose lengths live on the GPU together, as a decode loop uses
them: one captured step (tables grow, keys and values go to their slots, the
batch attends behind its shared prefix, tokens are drawn) is replayed, and
after every replay each stage is compared with its definition on what the stage
before it gave.  In between, requests are cut back (rejected drafts) and end,
and others take their pages, by the same operators outside the graph."""
import numpy as np
import pytest
import torch

from oracle import batch as oracle
from test_prefix_attention import check as check_attention

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu


def test_a_captured_step_replayed():
    requests, hq, hkv, d, vocab, prefix, width = 6, 8, 2, 64, 997, 70, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = 5 + requests * width
    k_pages, v_pages = (randn(pages, hkv, 16, d).to(torch.bfloat16) for _ in range(2))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    prefix_pages, free = order[:5].clone(), order[5:].clone()
    k_pages[prefix_pages[4].long(), :, 6:] = float("nan")  # past the prefix's end
    n_free, lens, status = ints([len(free)]), ints([0] * requests), ints([0])
    table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    embed = randn(vocab, (hq + 2 * hkv) * d).to(torch.bfloat16)
    head = randn(hq * d, vocab)
    tokens, u, one = ints(list(range(requests))), torch.rand(requests, generator=g, device="cuda"), ints([1] * requests)
    temperature, top_k = torch.full((requests,), 0.8, device="cuda"), ints([50, 0, 10, 1, 997, 3])
    stage = {}

    def step():
        slots, positions, cu = ta.extend_tables(lens, one, table, free, n_free, requests, position_base=prefix, status=status)
        x = embed[tokens.long()].reshape(requests, hq + 2 * hkv, d)
        ta.append_slots(x[:, hq:hq + hkv], x[:, hq + hkv:], slots, k_pages, v_pages, status=status)
        out, lse = ta.prefix_attention(x[:, :hq], k_pages, v_pages, table, lens, cu, prefix_pages, prefix, status=status)
        logits = out.float().reshape(requests, -1) @ head
        drawn, logprobs = ta.sample(logits, u, temperature, top_k, top_p=0.95)
        stage.update(slots=slots, positions=positions, x=x, out=out, lse=lse, logits=logits, drawn=drawn, logprobs=logprobs, cu=cu)
        tokens.copy_(drawn)

    state = [t.clone() for t in (lens, table, free, n_free, tokens)]
    step()  # once outside a graph, and its state put back
    for t, was in zip((lens, table, free, n_free, tokens), state):
        t.copy_(was)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy()  # noqa: E731
    for i in range(40):
        if i == 17:  # drafts of three requests are rejected, one request ends
            ta.extend_tables(lens, ints([-3, 0, -17, 0, -100, -1]), table, free, n_free, 0, status=status)
            assert lens.tolist() == [14, 17, 0, 17, 0, 16]
        u.copy_(torch.rand(requests, generator=g, device="cuda"))
        before = {n: t.clone() for n, t in dict(lens=lens, table=table, free=free, n_free=n_free, k=k_pages, v=v_pages).items()}
        graph.replay()
        torch.cuda.synchronize()
        want = oracle.extend_tables(before["lens"].tolist(), [1] * requests, before["table"].tolist(), before["free"].tolist(),
                                    before["n_free"].item(), requests, prefix)
        got = [stage["slots"], stage["positions"], stage["cu"], lens, table, free]
        assert [t.tolist() for t in got] == list(want[:6]) and n_free.item() == want[6]
        kv = oracle.append_slots(bits(stage["x"][:, hq:hq + hkv]), bits(stage["x"][:, hq + hkv:]), want[0], bits(before["k"]),
                                 bits(before["v"]))
        assert np.array_equal(bits(k_pages), kv[0]) and np.array_equal(bits(v_pages), kv[1])
        if i % 8 == 0 or i == 17:
            s = dict(q=stage["x"][:, :hq].cpu(), k=k_pages.cpu(), v=v_pages.cpu(), table=table.cpu(), lens=lens.cpu(),
                     cu_all=np.arange(requests + 1), pre=prefix_pages.cpu(), prefix=prefix, dtype="bf16")
            check_attention(s, stage["out"], stage["lse"])
        x, numbers = stage["logits"].cpu().numpy(), u.cpu().numpy()
        for r in range(requests):
            t, lp = oracle.sample(x[r], [numbers[r]], float(np.float32(0.8)), int(top_k[r]), float(np.float32(0.95)))[0]
            assert stage["drawn"][r].item() == t and abs(stage["logprobs"][r].item() - lp) <= 1e-5
    assert status.item() == 0
    # the tables' pages and the stack's are all pages behind the prefix, each once
    held = [table[b, j].item() for b in range(requests) for j in range(-(-int(lens[b]) // 16))]
    assert sorted(held + free[: n_free.item()].tolist()) == sorted(order[5:].tolist())
