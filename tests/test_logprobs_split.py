"""Rows of logits that several CTAs share: their sums and lists meet in one CTA's shared memory, whichever of
them starts or ends first.  Tolerances: test_logprobs.py."""
import pytest
import torch

from test_logprobs import check, logits, run

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,vocab", [("fp32", 8193), ("bf16", 16400), ("fp32", 50257), ("bf16", 262144)])
@pytest.mark.parametrize("rows", [1, 19, 57, 114, 225])
@pytest.mark.parametrize("top", [0, 5])
def test_the_same_again_and_again(top, rows, vocab, dtype):
    """The first parts of a row may be long done or not begun when the others' sums arrive."""
    x = logits(rows + vocab, rows, vocab, dtype).cuda()
    given = [[0, vocab - 1, vocab // 2]] * rows
    tokens = torch.tensor(given, dtype=torch.int32, device="cuda")
    first = run(x, given, 0.8, top)
    shown = [0, rows - 1]
    check(x[shown].cpu(), [given[r] for r in shown], 0.8, top, [g[shown] for g in first])
    # others' shared memory is left behind in the SMs in between
    other = torch.full((rows, vocab), 3.0, dtype=x.dtype, device="cuda")
    for _ in range(40):
        ta.token_logprobs(other, tokens, 0.8, top)
        again = ta.token_logprobs(x, tokens, 0.8, top)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_two_streams_at_once():
    """Clusters of two calls side by side: their CTAs start as places come free."""
    calls = [(logits(s, 60, 40000 + s, "bf16").cuda(), top) for s, top in ((1, 0), (2, 8))]
    want = [ta.token_logprobs(x, top=top) for x, top in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[ta.token_logprobs(x, top=top, stream=s) for _ in range(30)] for (x, top), s in zip(calls, streams)]
    torch.cuda.synchronize()
    for first, runs in zip(want, got):
        for again in runs:
            assert all(torch.equal(a, b) for a, b in zip(first[1:], again[1:]))
