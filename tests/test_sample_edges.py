"""Rows of logits at the edges of what sampling promises, against the
definition in float64 (`oracle.batch.sample`)."""
import math

import pytest
import torch

from test_sample import check, numbers

ta = pytest.importorskip("tree_structured_decode_gb300")

INF = float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab", [(3, 4000), (60, 8000), (3, 8000), (30, 30000), (3, 130000), (160, 70000)])
@pytest.mark.parametrize("masked", [True, False])
def test_top_k_ends_at_the_last_of_many_equal_logits(rows, vocab, masked):
    """1000 equal logits, top-k 1000, and a top-p that ends among them; rows of one, two and four CTAs."""
    g = torch.Generator().manual_seed(vocab)
    x = torch.full((rows, vocab), -INF) if masked else torch.randn((rows, vocab), generator=g) - 9
    for i in range(rows):
        x[i, torch.randperm(vocab, generator=g)[:1000]] = 0.5
    x = x.cuda()
    some = range(0, rows, max(1, rows // 3))
    for n, kw in enumerate([dict(top_p=0.75), dict(top_p=0.375), dict(top_p=1 - 2.0 ** -9, min_p=0.5), dict(top_p=0.0), {}]):
        for _ in range(3):
            check(x, numbers(n, rows, 5), rows=some, top_k=1000, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [60, 9000])
def test_infinity_is_above_the_largest_number(vocab):
    """+inf shares the row among its like, not with the largest finite number: its weight is exp(-inf)."""
    x = torch.randn((4, vocab), generator=torch.Generator().manual_seed(vocab)).cuda()
    most = torch.finfo(torch.float32).max
    x[0, 3], x[0, 40] = most, INF
    x[1, ::2], x[1, [5, 51]] = most, INF
    x[2, 7], x[2, 8:] = INF, most
    x[3, 2], x[3, 50] = most, -INF  # no infinity: the largest number has the row for itself
    for kw in (dict(temperature=0.0), {}, dict(top_k=3), dict(top_p=0.9), dict(min_p=0.3), dict(temperature=1e30, top_k=20, top_p=0.8)):
        check(x, numbers(6, 4, 7), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("top_k", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 1, 2 ** 40, -2 ** 32 + 1])
def test_a_top_k_of_any_size(top_k):
    """At or above the vocabulary, or not above 0: off, whatever its size."""
    x = torch.randn((3, 50), generator=torch.Generator().manual_seed(1)).cuda()
    want = ta.sample(x, numbers(2, 3, 40))
    assert all(torch.equal(a, b) for a, b in zip(want, ta.sample(x, numbers(2, 3, 40), top_k=top_k)))


@pytest.mark.gpu
@pytest.mark.parametrize("units", [0.3, 0.34, 0.66, 0.75, 1.4, 1.5, 2.3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_flat_tail_of_tiny_weights(units, dtype):
    """262143 equal weights of so many 2^-42: all rounded in one direction, by up to 0.67 units.  The token is right for a
    number within 262144 * 0.67 * 2^-42 of u's place (and one unit: the place is a whole number); below half a unit the tail
    is never drawn."""
    n = 262144
    x = torch.full((1, n), math.log(units * 2.0 ** -42))
    first = 1000
    x[0, first] = 0
    x = x.to(dtype).cuda()
    w = math.exp(x[0, 0].item())  # of the rounded logit
    u = 1 - torch.cat([2.0 ** -torch.arange(12, 25).float(), torch.arange(1, 90) * 2.0 ** -24])
    tokens, logprobs = ta.sample(x, u.reshape(1, -1).cuda())
    total, off = 1 + (n - 1) * w, (n * 0.67 + 1) * 2.0 ** -42
    before = lambda i: i * w if i <= first else 1 + (i - 1) * w  # noqa: E731
    for t, lp, place in zip(tokens[0].tolist(), logprobs[0].tolist(), (u.double() * total).tolist()):
        assert before(t) - off <= place <= before(t + 1) + off
        assert t == first or w * 2.0 ** 42 >= 0.5
        assert abs(lp - math.log((1 if t == first else w) / total)) <= 1e-5
    for kw in (dict(top_p=1 - 2.0 ** -22), dict(top_k=1), dict(top_k=5), dict(min_p=0.5)):
        got, _ = ta.sample(x, u.reshape(1, -1).cuda(), **kw)
        assert (got == first).all()


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [0.3, 1.0, 1e30])
def test_min_p_of_one_and_above(temperature):
    """Leaves the logits equal to the largest, all of them: any other weighs less than 1, at whatever temperature."""
    x = torch.randn((5, 700), generator=torch.Generator().manual_seed(3))
    for i in range(1, 5):
        x[i, torch.randperm(700, generator=torch.Generator().manual_seed(i))[: 3 ** i]] = x[i].max()
    x, u = x.cuda(), numbers(4, 5, 60)
    want, _ = check(x, u, 1.0, min_p=1.0)
    assert (x.gather(1, torch.from_numpy(want).long().cuda()) == x.amax(1, keepdim=True)).all()
    ties = (x == x.amax(1, keepdim=True)).sum(1, keepdim=True)
    for min_p in (1.0, 1.5, float("inf"), torch.full((5,), 3.0, device="cuda")):
        tokens, logprobs = ta.sample(x, u, temperature, min_p=min_p)
        assert (tokens.cpu().numpy() == want).all()
        assert (logprobs + ties.log()).abs().max() <= 1e-5
