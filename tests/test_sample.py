"""Sampling from given random numbers, against its definition in float64.

Tokens are equal: the kernel's weights are exact to 2^-42 of the largest, so a
token could differ only where u times the total lies within about the number
of tokens times 2^-42 of a border, which none of these fixed inputs does.
logprob: th and tl carry the exponent to far below 2^-24, log2 of the total and
the sums of the pair round at 2^-24 of numbers up to 45 (and log2f by one more
step): 2^-24 * 45 * 3 + the last product's 2^-24 of the result, below 1e-5."""
import math

import numpy as np
import pytest
import torch

from oracle import batch as oracle

ta = pytest.importorskip("tree_structured_decode_gb300")
from tree_structured_decode_gb300 import _abi  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def check(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=None, **kw):
    """The call's result against the oracle, row by row (all, or the ones given)."""
    tokens, logprobs = ta.sample(logits, u, temperature, top_k, top_p, min_p, **kw)
    assert tokens.shape == u.shape and tokens.dtype == torch.int32 and logprobs.dtype == torch.float32
    x, numbers = logits.float().cpu().numpy(), u.cpu().numpy().reshape(len(u), -1)
    tokens, logprobs = tokens.cpu().numpy().reshape(numbers.shape), logprobs.cpu().numpy().reshape(numbers.shape)
    at = lambda v, i: float(v[i]) if torch.is_tensor(v) else v  # noqa: E731
    for i in range(len(x)) if rows is None else rows:
        want = oracle.sample(x[i], numbers[i], at(temperature, i), int(at(top_k, i)), at(top_p, i), at(min_p, i))
        assert tokens[i].tolist() == [w[0] for w in want], i
        for got, (_, w) in zip(logprobs[i], want):
            assert math.isnan(got) if math.isnan(w) else abs(got - w) <= 1e-5, i
    return tokens, logprobs


def rows_of(seed, rows, vocab, dtype="fp32", spread=3.0, stride=None):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn((rows, stride or vocab), generator=g)
    return x.to(TYPES[dtype]).cuda()[:, :vocab]


def numbers(seed, *shape):
    return torch.rand(shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab,stride", [(1, 1, 1), (3, 2, 2), (5, 31, 33), (40, 33, 40), (7, 1000, 1001), (3, 8193, 8200),
                                               (2, 50257, 50257)])
def test_filters(rows, vocab, stride, dtype):
    x = rows_of(vocab, rows, vocab, dtype, stride=stride)
    for n, kw in enumerate([{}, dict(temperature=0.7, top_k=5), dict(temperature=1.6, top_p=0.8), dict(min_p=0.05),
                            dict(temperature=0.9, top_k=40, top_p=0.95, min_p=0.02), dict(top_k=1), dict(top_p=0.0),
                            dict(top_k=vocab // 2 + 1, top_p=0.999)]):
        check(x, numbers(n, rows, 1 + n % 3), **kw)


@pytest.mark.gpu
def test_parameters_of_each_row():
    x = rows_of(1, 60, 3000)
    g = np.random.default_rng(2)
    put = lambda v, t: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    check(x, numbers(3, 60, 2), put(g.choice([0, -1, 0.3, 1, 2.5], 60), torch.float32),
          put(g.choice([0, -3, 1, 7, 2999, 3000, 5000], 60), torch.int32), put(g.choice([-0.1, 0, 0.3, 0.9, 1, 2], 60), torch.float32),
          put(g.choice([-1, 0, 0.001, 0.3, 1, 2], 60), torch.float32))


@pytest.mark.gpu
def test_ties():
    """Equal logits: by index, and a filter that ends among them keeps the first ones."""
    same = torch.zeros((1, 4000), device="cuda")
    u = torch.arange(4000, device="cuda").reshape(1, -1) / 4096
    check(same, u)
    for k in (1, 2, 999, 3999):
        tokens, _ = check(same, u, top_k=k)
        assert tokens.max() < k
    check(same, u, top_p=0.5)
    tokens, _ = check(same, u, top_p=0.25)
    assert tokens.max() < 1000
    x = torch.tensor([[0.0, -0.0, 1.0, -0.0, 0.0, 1.0]], device="cuda")
    for k in range(1, 6):
        check(x, numbers(k, 1, 50), top_k=k)
    few = torch.randint(0, 4, (6, 5000), generator=torch.Generator().manual_seed(8)).float().cuda()
    for kw in (dict(top_k=700), dict(top_k=1300, top_p=0.9), dict(top_p=0.6), dict(min_p=0.2), dict(top_p=0.99, temperature=0.4)):
        check(few, numbers(9, 6, 20), **kw)


@pytest.mark.gpu
def test_masks_infinities_and_nan():
    x = rows_of(4, 9, 700)
    inf = float("inf")
    x[0, :] = -inf                # nothing left
    x[1, :699] = -inf             # one left
    x[2, 5], x[2, 9] = inf, inf   # they share the row
    x[3, 600] = float("nan")
    x[4, ::2] = -inf
    x[5, 3] = inf
    x[6] *= 1e30                  # differences beyond the range of exp
    x[7] = torch.finfo(torch.float32).max
    x[7, 1::2] = torch.finfo(torch.float32).min
    for kw in ({}, dict(top_k=2), dict(top_p=0.7), dict(min_p=0.5), dict(temperature=0.0), dict(temperature=1e-30), dict(temperature=1e-45),
               dict(temperature=1e30, top_k=100, top_p=0.9)):
        check(x, numbers(5, 9, 4), **kw)
    tokens, logprobs = ta.sample(x, numbers(5, 9))
    assert tokens[[0, 3]].tolist() == [-1, -1] and logprobs[[0, 3]].isnan().all()


@pytest.mark.gpu
def test_numbers_at_and_past_the_ends():
    x = rows_of(6, 1, 50)
    x[0, 45:] = -float("inf")
    ends = torch.tensor([[0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, float("nan")]], device="cuda")
    tokens, _ = ta.sample(x, ends)
    assert tokens[0, [0, 4, 5]].tolist() == [0, 0, 0] and tokens[0, [2, 3]].tolist() == [44, 44]


@pytest.mark.gpu
@pytest.mark.parametrize("vocab,dtype", [(131072, "fp32"), (262144, "bf16"), (100003, "fp16")])
def test_large_rows(vocab, dtype):
    """Rows of several CTAs, few and many of them; filters that keep few, many and nearly all tokens."""
    x = rows_of(vocab, 2, vocab, dtype)
    for n, kw in enumerate([{}, dict(top_k=50, top_p=0.9), dict(top_p=0.9), dict(top_p=0.9999), dict(top_k=vocab - 7), dict(min_p=1e-6)]):
        check(x, numbers(n, 2, 3), **kw)
    many = x.repeat(120, 1)
    u = numbers(77, 240)
    check(many, u, temperature=0.8, top_p=0.95, rows=range(0, 240, 61))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 60, 400])
def test_filters_that_end_far_below_the_largest(rows):
    """Steep rows, where a filter's end lies past 2^-16 and 2^-24 of the largest weight, and rows of few distinct values, whose
    bins hold thousands."""
    x = rows_of(31, rows, 9000, spread=6.0)
    x[rows // 2] = (x[rows // 2] / 4).round()
    some = range(0, rows, max(1, rows // 5))
    for n, kw in enumerate([dict(top_k=7000), dict(top_k=7000, top_p=1 - 2.0 ** -23), dict(top_p=1 - 2.0 ** -24),
                            dict(top_p=1 - 2.0 ** -20, temperature=2.0), dict(top_k=8999, temperature=0.5), dict(top_p=0.9999, min_p=1e-7)]):
        check(x, numbers(n, rows, 2), rows=some, **kw)


@pytest.mark.gpu
def test_many_draws_follow_the_weights():
    """All of a row's tokens come, each as often as its share of evenly spread numbers says (to one)."""
    x = rows_of(10, 1, 300, spread=1.0)
    n = 1 << 16
    u = ((torch.arange(n, device="cuda") + 0.5) / n).reshape(1, -1)
    tokens, _ = ta.sample(x, u)
    share = torch.softmax(x.double()[0], 0)
    assert (tokens[0].bincount(minlength=300) - share * n).abs().max() <= 1


@pytest.mark.gpu
def test_streams_graphs_and_views():
    x = rows_of(11, 20, 9000, stride=9010)
    u = numbers(12, 20, 2)
    want = ta.sample(x, u, top_k=30)
    assert all(torch.equal(a, b) for a, b in zip(want, ta.sample(x.contiguous(), u, top_k=30)))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = ta.sample(x, u, top_k=30, stream=stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = ta.sample(x, u, top_k=30)
    u.copy_(u.flip(0))
    graph.replay()
    stream.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    assert all(torch.equal(a, b) for a, b in zip(kept, ta.sample(x, u, top_k=30)))
    tokens, logprobs = ta.sample(x[:0], u[:0])
    assert tokens.shape == (0, 2)
    assert ta.sample(x, u[:, :0])[0].shape == (20, 0)


# ------------------------------------------------------------- refusals (no GPU)
def _sample(**kw):
    a = dict(logits=64, stride=100, dtype=2, rows=2, vocab=100, u=64, draws=1, t=None, t0=1.0, k=None, k0=0, p=None, p0=1.0,
             m=None, m0=0.0, tokens=64, logprobs=None, stream=None)
    a.update(kw)
    return _abi.load_library().tree_attn_sample(*a.values())


@pytest.mark.parametrize("kw,name", [
    (dict(logits=None), "INVALID_ARG"), (dict(u=None), "INVALID_ARG"), (dict(tokens=None), "INVALID_ARG"),
    (dict(rows=-1), "INVALID_ARG"), (dict(vocab=0), "INVALID_ARG"), (dict(draws=-1), "INVALID_ARG"),
    (dict(stride=99), "INVALID_ARG"), (dict(dtype=3), "UNSUPPORTED"), (dict(vocab=262145, stride=262145), "UNSUPPORTED"),
    (dict(rows=1 << 28), "UNSUPPORTED"), (dict(logits=66), "ALIGNMENT"), (dict(u=65), "ALIGNMENT"), (dict(m=66), "ALIGNMENT")])
def test_refusals(kw, name):
    assert _abi.STATUS_NAMES[_sample(**kw)] == "TA_ERR_" + name


def test_nothing_to_draw_is_done_at_once():
    assert _sample(rows=0) == _abi.TA_OK and _sample(draws=0) == _abi.TA_OK


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="CUDA"):
        ta.sample(torch.zeros(1, 4), torch.zeros(1))


@pytest.mark.gpu
def test_wrong_tensors_are_refused():
    x, u = torch.zeros((2, 8), device="cuda"), torch.zeros(2, device="cuda")
    for a, kw in (((x.double(), u), {}), ((x.t(), u), {}), ((x[0], u), {}), ((x, u.double()), {}), ((x, u[:1]), {}),
                  ((x, u.cpu()), {}), ((x, u), dict(top_k=u)), ((x, u), dict(temperature=u[:1])), ((x, u), dict(min_p=u.double()))):
        with pytest.raises(ValueError):
            ta.sample(*a, **kw)


def test_the_definition_on_rows_worked_out_by_hand():
    """Weights 4, 2, 1, 1 (logits ln 4, ln 2, 0, 0) in index order 2, 4, 1, 1."""
    row = [math.log(2), math.log(4), 0.0, 0.0]
    u = [0.0, 0.249, 0.251, 0.74, 0.76, 0.874, 0.876, 0.999]
    tok = lambda **kw: [t for t, _ in oracle.sample(row, u, **kw)]  # noqa: E731
    assert tok() == [0, 0, 1, 1, 2, 2, 3, 3]
    assert tok(top_k=1) == [1] * 8
    assert tok(top_k=3) == [0, 0, 0, 1, 1, 2, 2, 2]          # 2/7, 6/7
    assert tok(top_p=0.7) == [0, 0, 0, 1, 1, 1, 1, 1]        # 4 + 2 of 8
    assert tok(min_p=0.3) == [0, 0, 0, 1, 1, 1, 1, 1]
    assert tok(temperature=0) == [1] * 8
    assert oracle.sample(row, [0.9], top_k=3)[0][1] == pytest.approx(math.log(1 / 7))
