"""The likeliest tokens where token 0 is the last of the list so far and a later logit is one step above it.
Tolerances: test_logprobs.py."""
import math

import pytest
import torch

from test_logprobs import check, run

ta = pytest.importorskip("tree_structured_decode_gb300")

pytestmark = pytest.mark.gpu


def rows_of(vocab, top, low, later, at):
    """Bulk `bulk`, token 0 at `low` with top - 1 larger ones beside it, a later logit of `later`."""
    x = torch.full((vocab,), low - 11 if math.isfinite(low - 11) else -1.0)
    x[:top] = low + 0.5 if low + 0.5 > low else math.inf
    x[0] = low
    x[at] = later
    return x


# one CTA a row, of 256 threads and of 128; a row over several
@pytest.mark.parametrize("copies,vocab", [(300, 32000), (700, 9000), (1, 262144), (60, 100000)])
@pytest.mark.parametrize("top", [1, 2, 7, 64])
@pytest.mark.parametrize("low", [1.0, -1.0, 0.0, 5.0, 1e-30])
def test_one_step_above_token_0(low, top, copies, vocab):
    later = float(torch.nextafter(torch.tensor(low), torch.tensor(math.inf)))
    at = 6000
    x = torch.stack([rows_of(vocab, top, low, later, at), rows_of(vocab, top, low, low, at)])
    masked = torch.full((vocab,), -math.inf)  # the first logits leave the list short of its k
    masked[: top] = x[0, : top]
    masked[5000], masked[6100], masked[8500] = low - 1, low - 2, later
    x = torch.cat([x, masked[None]])
    given = [[0, at]] * len(x)
    got = run(x.repeat(copies, 1), given * copies, 1.0, top)
    check(x, given, 1.0, top, [g[: len(x)] for g in got])
    for g in got:
        assert torch.equal(g.reshape(copies, -1), g[: len(x)].reshape(1, -1).expand(copies, -1))


@pytest.mark.parametrize("copies", [1, 300])
def test_the_largest_finite_value_and_an_infinite_one(copies):
    big = torch.finfo(torch.float32).max
    x = torch.zeros((2, 40000))
    x[0, 0], x[0, 9000] = big, math.inf
    x[1, 0], x[1, 1], x[1, 9000] = -big, 4.0, float(torch.nextafter(torch.tensor(-big), torch.tensor(0.0)))
    x[1, 2:9000], x[1, 9001:] = -math.inf, -math.inf
    given = [[0, 9000]] * 2
    for top in (1, 2, 3):
        got = run(x.repeat(copies, 1), given * copies, 1.0, top)
        check(x, given, 1.0, top, [g[:2] for g in got])


@pytest.mark.parametrize("copies", [1, 300])
def test_no_temperature_finds_the_largest(copies):
    x = torch.full((1, 40000), -math.inf)
    x[0, 0], x[0, 1], x[0, 2] = 1.0, 0.5, 0.25
    x[0, 4500], x[0, 9000] = 0.5, float(torch.nextafter(torch.tensor(1.0), torch.tensor(2.0)))
    for top in (0, 1):
        got = run(x.repeat(copies, 1), [[0, 9000]] * copies, [0.0] * copies, top)
        check(x, [[0, 9000]], 0.0, top, [g[:1] for g in got])
